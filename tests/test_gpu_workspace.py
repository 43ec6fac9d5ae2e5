"""Workspaces a call makes for itself, on a stream other than the current one,
and calls whose longest length is zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

S, HQ, HKV, D, BS, N = 3, 8, 2, 64, 16, 1000


def _inputs(n=N):
    g = torch.Generator(device="cuda").manual_seed(1)
    nblk = -(-N // BS)
    NB = S * nblk + 1
    tables = (torch.randperm(NB - 1, device="cuda", generator=g) + 1)[:S * nblk].view(S, nblk).int()
    t = torch.arange(N, device="cuda")
    slots = tables[:, t // BS] * BS + (t % BS).int()
    k, v = (torch.randn(NB, BS, HKV, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    k4, v4 = (pkv.make_kv4_cache(NB, BS, HKV, D) for _ in range(2))
    pkv.paged_kv4_write(k.flatten(0, 1), v.flatten(0, 1), k4, v4, torch.arange(NB * BS, device="cuda"), BS)
    lens = torch.tensor([n, n // 2, n // 3], dtype=torch.int32, device="cuda")
    q = torch.randn(S, HQ, D, device="cuda", generator=g).bfloat16()
    starts = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    scores = torch.zeros(S, N, device="cuda")
    sc = D ** -0.5
    return {
        "decode": lambda o, m, **kw: pkv.paged_attention_decode(o, q, k, v, tables, lens, m, sc, **kw),
        "token": lambda o, m, **kw: pkv.token_attention_decode(o, q, k, v, slots, lens, m, sc, **kw),
        "prefill": lambda o, m, **kw: pkv.paged_attention_prefill(o, q, k, v, tables, lens, starts, min(1, m), m, sc,
                                                                  **kw),
        "window": lambda o, m, **kw: pkv.paged_attention_decode_window(o, q, k, v, tables, lens, m, sc, 700, 4, **kw),
        "prefill_window": lambda o, m, **kw: pkv.paged_attention_prefill_window(o, q, k, v, tables, lens, starts,
                                                                                min(1, m), m, sc, 700, 4, **kw),
        "kv4": lambda o, m, **kw: pkv.paged_attention_decode_kv4(o, q, k4, v4, tables, lens, m, sc, BS, **kw),
        "scored": lambda o, m, **kw: pkv.token_attention_decode_scored(o, q, k, v, slots, lens, scores, m, sc, **kw),
    }, q


@pytest.mark.parametrize("name", ["decode", "token", "prefill", "window", "prefill_window", "kv4", "scored"])
@pytest.mark.parametrize("raw", [False, True])
def test_own_workspace_on_another_stream(name, raw):
    """The current stream is busy, and its allocator holds blocks full of ones: the call on the side stream still
    finds its workspace zeroed."""
    calls, q = _inputs()
    want = calls[name](torch.empty_like(q), N, partition_size=128)
    got = torch.empty_like(q)
    side = torch.cuda.Stream()
    junk = [torch.full((1 << 16 << i,), 0xFF, dtype=torch.uint8, device="cuda") for i in range(8)]
    torch.cuda.synchronize()
    del junk
    torch.cuda._sleep(20_000_000)
    calls[name](got, N, partition_size=128, stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert torch.equal(got.cpu(), want.cpu())


@pytest.mark.parametrize("name", ["window", "kv4", "scored"])
def test_longest_length_zero(name):
    """max 0: every length is clamped to it and every output row is zero."""
    calls, q = _inputs()
    out = calls[name](torch.full_like(q, 7.0), 0)
    assert torch.equal(out, torch.zeros_like(q))


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3", "kv4"])
@pytest.mark.parametrize("d,part", [(64, 64), (128, 64), (128, 128), (128, 32)])
def test_small_and_large_launches_agree(kind, d, part):
    """Few (sequence, head set) pairs, whose partitions one launch merges, and the same sequences among many, whose
    partitions a second launch merges: the same bits, with lengths from none to all partitions."""
    lens, few, many, hkv = [0, 1, part, part + 1, 3 * part - 5, 4 * part], 6, 84, 2
    n = max(lens)
    nblk = -(-n // BS)
    g = torch.Generator(device="cuda").manual_seed(3)
    tables = torch.randperm(few * nblk, device="cuda", generator=g).view(few, nblk).int()
    k, v = (torch.randn(few * nblk, BS, hkv, d, device="cuda", generator=g) for _ in range(2))
    if kind == "kv4":
        kc, vc = (pkv.make_kv4_cache(few * nblk, BS, hkv, d) for _ in range(2))
        pkv.paged_kv4_write(k.flatten(0, 1), v.flatten(0, 1), kc, vc, torch.arange(few * nblk * BS, device="cuda"), BS)
    else:
        kc, vc = (x.to({"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kind]) for x in (k, v))
    q = torch.randn(few, 10, d, device="cuda", generator=g).bfloat16()
    c = torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = []
    for copies in (1, many // few):
        qs, ts, cs = (x.repeat(copies, *[1] * (x.dim() - 1)) for x in (q, tables, c))
        out = torch.full_like(qs, float("nan"))
        if kind == "kv4":
            pkv.paged_attention_decode_kv4(out, qs, kc, vc, ts, cs, n, d ** -0.5, BS, partition_size=part)
        else:
            pkv.paged_attention_decode_window(out, qs, kc, vc, ts, cs, n, d ** -0.5, n, 0, partition_size=part)
        outs.append(out)
    assert not outs[0].isnan().any() and (outs[0][0] == 0).all()
    for i in range(many // few):
        assert torch.equal(outs[1][i * few:(i + 1) * few], outs[0])
