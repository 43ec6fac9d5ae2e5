"""Lengths, starts and slots that the kernel before a call writes: a launch may
begin while that kernel runs, and reads none of them before it has ended."""
import pytest
import torch

from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

BF = torch.bfloat16


def queued(step, kept, repeats=8):
    """step(i) behind kernels that clear and then fill the tensors that `kept` maps to their contents."""
    torch.cuda.synchronize()
    for i in range(repeats):
        for t, _ in kept:
            t.zero_()
        for t, x in kept:
            t.copy_(x)
        step(i)
    torch.cuda.synchronize()


# small batches go through the windowed decode, larger ones through the plain one
@pytest.mark.parametrize("groups,windowed", [([(304, [305, 344, 304, 400])], True), ([(304, [500 + 7 * i for i in range(170)])], False),
                                             ([(2048, [2050, 3000, 9000])], False)])
def test_shared_decode_on_its_own(groups, windowed):
    c = Case(groups, 12, 2, 128, 16, seed=41)
    S, Hq, Hkv, d = c.shape
    size = pkv.shared_workspace_size(S, 1, Hq, Hkv, d, 16, *c.bounds)
    plain = pkv.decode_workspace_size(S, Hq, Hkv, d, 16, c.bounds[0])
    assert size == (pkv.decode_window_workspace_size(S, Hq, Hkv, d, 16, c.bounds[0], c.bounds[0]) if windowed else plain)
    ws = pkv.make_shared_workspace(S, 1, Hq, Hkv, d, 16, *c.bounds)
    want = c.run(sharing="auto", workspace=ws)
    c.check(want)
    outs = [torch.zeros_like(want) for _ in range(8)]

    def step(i):
        pkv.paged_attention_decode_shared(outs[i], c.q, c.kc, c.vc, c.tables, c.n, c.starts, c.shared, *c.bounds, c.scale,
                                          workspace=ws)

    queued(step, [(t, t.clone()) for t in (c.n, c.starts, c.shared)])
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("ql", [[5, 40, 3], [300, 1, 520]])
def test_query_chunks(window, ql):
    g = torch.Generator(device="cuda").manual_seed(42)
    n, bs, Hq, Hkv, d = [700, 41, 900], 16, 12, 2, 128
    kc, vc = (torch.randn(120, bs, Hkv, d, device="cuda", generator=g).to(BF) for _ in range(2))
    tables = torch.randperm(120, device="cuda", generator=g)[:3 * 40].view(3, 40).int()
    tables = torch.cat((tables, tables.flip(1)), 1).contiguous()
    ql = [min(a, b) for a, b in zip(ql, n)]
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, ql[0], ql[0] + ql[1], sum(ql)], dtype=torch.int32, device="cuda")
    q = torch.randn(sum(ql), Hq, d, device="cuda", generator=g).to(BF)

    def one(out):
        if window:
            pkv.paged_attention_prefill_window(out, q, kc, vc, tables, lens, starts, max(ql), 960, d ** -0.5, window, 4)
        else:
            pkv.paged_attention_prefill(out, q, kc, vc, tables, lens, starts, max(ql), 960, d ** -0.5)

    want = torch.zeros_like(q)
    one(want)
    outs = [torch.zeros_like(q) for _ in range(8)]
    queued(lambda i: one(outs[i]), [(lens, lens.clone()), (starts, starts.clone())])
    assert want.abs().sum() > 0 and all(torch.equal(o, want) for o in outs)


def test_slots_of_a_4_bit_write():
    g = torch.Generator(device="cuda").manual_seed(43)
    bs, Hkv, d, T = 16, 2, 128, 50
    k, v = (torch.randn(T, Hkv, d, device="cuda", generator=g).to(BF) for _ in range(2))
    slots = torch.randperm(10 * bs, device="cuda", generator=g)[:T]
    shape = (10, Hkv, pkv.kv4_block_bytes(bs, Hkv, d) // Hkv)
    want = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pkv.paged_kv4_write(k, v, *want, slots, bs)
    pools = [[torch.zeros_like(w) for w in want] for _ in range(8)]
    kept = slots.clone()
    torch.cuda.synchronize()
    for p in pools:
        slots.fill_(-1)
        slots.copy_(kept)
        pkv.paged_kv4_write(k, v, *p, slots, bs)
    torch.cuda.synchronize()
    for p in pools:
        for a, b in zip(p, want):
            assert torch.equal(a, b)
