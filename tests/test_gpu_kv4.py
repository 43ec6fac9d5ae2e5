"""The 4-bit cache on the GPU: write and read bit for bit against the
definition's fp32 operations, the decode against 64 bits over the values the
cache stands for."""
import numpy as np
import pytest
import torch

from tests import plain64 as P64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv


def _rows(T, Hkv, d, dtype, seed):
    """Rows with the groups that matter: ordinary, constant, huge, tiny,
    infinite and NaN ones."""
    x = np.random.default_rng(seed).standard_normal((T, Hkv, d)).astype(np.float32)
    odd = [lambda r: np.full_like(r, 1.2345), lambda r: r * 0, lambda r: r * 1e6, lambda r: r * 1e-6,
           lambda r: np.where(np.arange(r.size) == 3, np.inf, r), lambda r: np.where(np.arange(r.size) == 9, -np.inf, r),
           lambda r: np.where(np.arange(r.size) == 31, np.nan, r), lambda r: r * 1e-3 + 100]
    for i in range(T):
        x[i, i % Hkv, 32 * (i % (d // 32)):][:32] = odd[i % len(odd)](x[i, i % Hkv, 32 * (i % (d // 32)):][:32])
    t = torch.from_numpy(x).cuda().to(dtype)
    return t, t.float().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,Hkv,d,bs", [(1, 1, 64, 16), (37, 2, 128, 16), (100, 3, 64, 32), (333, 8, 128, 32)])
@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.37, 2.5), (1e-30, 1e30), (1e-40, 3e38)])
def test_write_and_read(dtype, T, Hkv, d, bs, scales):
    NB = -(-T // bs) + 3
    key, k32 = _rows(T, Hkv, d, dtype, 1)
    val, v32 = _rows(T, Hkv, d, dtype, 2)
    rng = np.random.default_rng(3)
    slots = rng.permutation(NB * bs)[:T].astype(np.int64)
    slots[T // 2] = -1 if T > 1 else slots[0]              # skipped
    kc, vc = (torch.full_like(pkv.make_kv4_cache(NB, bs, Hkv, d), 0xA5) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    pkv.paged_kv4_write(key, val, kc, vc, sl, bs, *scales, err_word=err)
    ko, vo = torch.full((2, T, Hkv, d), 9.0, device="cuda")
    pkv.paged_kv4_read(ko, vo, kc, vc, sl, bs, *scales, err_word=err)
    assert int(err) == 0
    for got, x, by in ((ko, k32, scales[0]), (vo, v32, scales[1])):
        want = P64.kv4_values(x, by)
        want[slots < 0] = 9.0
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    # bf16 out: the same values rounded once
    kb, vb = torch.zeros((2, T, Hkv, d), device="cuda", dtype=torch.bfloat16)
    pkv.paged_kv4_read(kb, vb, kc, vc, sl, bs, *scales)
    live = torch.from_numpy(slots >= 0).cuda()
    for a, b in ((kb, ko), (vb, vo)):
        assert torch.equal(torch.nan_to_num(a[live]), torch.nan_to_num(b[live].bfloat16()))
    # the documented places, and the untouched slots' bytes
    kn, vn = kc.cpu().numpy(), vc.cpu().numpy()
    blocks = sorted({int(s) // bs for s in slots if s >= 0})[:4]
    for b in blocks:
        for h in range(Hkv):
            for cache, x, by, isv in ((kn, k32, scales[0], False), (vn, v32, scales[1], True)):
                got = P64.kv4_block(cache, b, h, bs, d, isv)
                for i, s in enumerate(slots):
                    if s >= 0 and s // bs == b:
                        want = P64.kv4_values(x[i, h], by).astype(np.float64)
                        # the call takes the scale as fp32 and rounds the product to fp32 (subnormal, or past its range)
                        with np.errstate(over="ignore"):
                            val = (got[s % bs] * np.float64(np.float32(by))).astype(np.float32).astype(np.float64)
                        np.testing.assert_allclose(val, want, rtol=2.0 ** -22, atol=2.0 ** -148, equal_nan=True)
    fresh = np.setdiff1d(np.arange(NB * bs), slots)
    for b in sorted({int(s) // bs for s in fresh})[:4]:
        ref = np.full((1, 1, kn.shape[2]), 0xA5, np.uint8)
        for cache, isv in ((kn, False), (vn, True)):
            want = P64.kv4_block(ref, 0, 0, bs, d, isv)
            got = P64.kv4_block(cache, b, 0, bs, d, isv)
            rows = [s % bs for s in fresh if s // bs == b]
            np.testing.assert_array_equal(got[rows], want[rows])


def test_consecutive_tokens_of_one_call_and_of_single_calls_give_the_same_bytes():
    """A prompt written at once, from an odd position, and token by token."""
    for d, bs, Hkv in ((128, 16, 2), (64, 32, 3)):
        T, first = 83, 5
        key, _ = _rows(T, Hkv, d, torch.bfloat16, 5)
        val, _ = _rows(T, Hkv, d, torch.bfloat16, 6)
        order = torch.randperm(12, device="cuda")
        pos = torch.arange(first, first + T, device="cuda")
        slots = order[pos // bs] * bs + pos % bs
        a = [torch.zeros_like(pkv.make_kv4_cache(12, bs, Hkv, d)) for _ in range(2)]
        b = [torch.zeros_like(x) for x in a]
        pkv.paged_kv4_write(key, val, *a, slots, bs)
        for i in range(T):
            pkv.paged_kv4_write(key[i:i + 1], val[i:i + 1], *b, slots[i:i + 1].clone(), bs)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_slots_are_reported_and_touch_nothing():
    key, _ = _rows(3, 2, 128, torch.float32, 7)
    kc, vc = (pkv.make_kv4_cache(4, 16, 2, 128) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([64, -5, 1 << 40], device="cuda")
    pkv.paged_kv4_write(key, key, kc, vc, slots, 16, err_word=err)
    assert int(err) == 3 and not kc.any() and not vc.any()
    err.zero_()
    out = torch.full_like(key, 4.0)
    pkv.paged_kv4_read(out, out.clone(), kc, vc, slots, 16, err_word=err)
    assert int(err) == 3 and (out == 4).all()


def _decode_case(Hq, Hkv, d, bs, lens, window, sinks, part, seed=1, scales=(0.5, 2.0), scale=None):
    """The pool is written by the library; slots no query sees then get
    codes, scales and zeros of NaN, unseen blocks' entries go out of range."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nblk = [-(-n // bs) for n in lens]
    NB, MB = sum(nblk) + 1, max(max(nblk), 1)
    order = torch.randperm(NB, device="cuda", generator=g)
    kc, vc = (torch.full_like(pkv.make_kv4_cache(NB, bs, Hkv, d), 0xFF) for _ in range(2))   # fp16 0xffff: NaN
    tables = torch.full((len(lens), MB), -7, dtype=torch.int32, device="cuda")
    dense, at = [], 0
    for s, n in enumerate(lens):
        ids = order[at:at + nblk[s]]
        at += nblk[s]
        seen = P64.window_seen(n, n - 1, window, sinks)
        t = torch.nonzero(seen).flatten()
        k, v = torch.randn(2, n, Hkv, d, device="cuda", generator=g)
        slots = ids[t // bs] * bs + t % bs
        pkv.paged_kv4_write(k[t], v[t], kc, vc, slots, bs, *scales)
        for b in torch.unique(t // bs).tolist():
            tables[s, b] = ids[b]
        ko, vo = torch.zeros(2, n, Hkv, d, device="cuda")
        kr, vr = torch.empty(2, t.numel(), Hkv, d, device="cuda")
        pkv.paged_kv4_read(kr, vr, kc, vc, slots, bs, *scales)
        ko[t], vo[t] = kr, vr
        dense.append((ko, vo, seen))
    q = torch.randn(len(lens), Hq, d, device="cuda", generator=g).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, err = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    mx, scale = max(lens), d ** -0.5 if scale is None else scale
    ws = pkv.make_window_workspace(len(lens), Hq, Hkv, d, bs, mx, window, sinks, part)
    pkv.paged_attention_decode_kv4(out, q, kc, vc, tables, n, mx, scale, bs, window, sinks, *scales,
                                   partition_size=part, workspace=ws, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for s, (k, v, seen) in enumerate(dense):
        o, _, mix, reach = P64.attend(q[s], k, v, seen, scale)
        if not seen.any():
            assert (out[s] == 0).all()
            continue
        # weights rounded to fp16 and again after the group's scale; the zeros enter apart from the
        # codes, so magnitudes are those of scale * code and zero, at most four times the largest value;
        # fp16 products below 2^-14 are off by 2^-25 (times the code, 15)
        top = 4 * float(v.abs().max())
        few = int(seen.sum()) * 2.0 ** -25 * (15 * scales[1] + top)
        bound = P64.out_bound(o, mix, 4 * reach, d, 2.0 ** -8, 2.0 ** -8, few) + 2 * 2.0 ** -11 * top
        P64.assert_within(out[s], o, bound, f"sequence {s} of {lens[s]}")
    return out


LENS = [0, 1, 15, 16, 17, 37, 300, 1000, 2049]


@pytest.mark.parametrize("shape", [(4, 2, 64, 16), (12, 2, 128, 16), (28, 4, 128, 32), (10, 1, 64, 32), (3, 3, 128, 16),
                                   (64, 8, 128, 16)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (17, 33), (999, 5)])
def test_decode(shape, window, sinks):
    _decode_case(*shape, LENS, window, sinks, 0)


@pytest.mark.parametrize("part", [-1, 16, 32, 48, 64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (777, 20)])
def test_decode_partitions(part, window, sinks):
    _decode_case(16, 2, 128, 16, LENS, window, sinks, part)
    _decode_case(8, 2, 64, 32, [5000, 1, 700], window, sinks, part if part % 32 == 0 else -1)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_decode_with_other_logit_scales(scale):
    """Negative (the smallest product weighs most), zero (every token weighs the same), and large."""
    _decode_case(12, 2, 128, 16, [1, 100, 1500], 0, 0, 128, scale=scale)
    _decode_case(7, 1, 64, 32, [33, 700], 100, 5, 0, scale=scale)


def test_offsets_past_32_bits():
    """Pools of more than 2^32 bytes: write, read and decode in their last blocks."""
    bs, Hkv, d, Hq, n = 16, 8, 128, 16, 300
    NB = (1 << 32) // (Hkv * 1280) + 1000
    kc, vc = (pkv.make_kv4_cache(NB, bs, Hkv, d) for _ in range(2))
    assert kc.numel() > 1 << 32
    pos = torch.arange(n, device="cuda")
    ids = NB - 1 - torch.arange(-(-n // bs), device="cuda")
    slots = ids[pos // bs] * bs + pos % bs
    k, v = torch.randn(2, n, Hkv, d, device="cuda")
    pkv.paged_kv4_write(k, v, kc, vc, slots, bs)
    ko, vo = torch.zeros(2, n, Hkv, d, device="cuda")
    pkv.paged_kv4_read(ko, vo, kc, vc, slots, bs)
    np.testing.assert_array_equal(ko.cpu().numpy(), P64.kv4_values(k.cpu().numpy(), 1.0))
    assert not kc[:1000].any() and not vc[:1000].any()
    q = torch.randn(1, Hq, d, device="cuda").bfloat16()
    out = torch.empty_like(q)
    pkv.paged_attention_decode_kv4(out, q, kc, vc, ids.int()[None].contiguous(),
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), n, 0.1, bs)
    o, _, mix, reach = P64.attend(q[0], ko, vo, torch.ones(n, dtype=torch.bool, device="cuda"), 0.1)
    P64.assert_within(out[0], o, P64.out_bound(o, mix, 4 * reach, d, 2.0 ** -8, 2.0 ** -8) + 2.0 ** -7)


def test_a_nan_reaches_its_head_only():
    """A NaN written to one value of one token of K/V head 0 makes that head's queries NaN, and no others."""
    bs, Hkv, d, Hq, n = 16, 2, 64, 8, 100
    kc, vc = (pkv.make_kv4_cache(14, bs, Hkv, d) for _ in range(2))
    k, v = torch.randn(2, 2 * 7 * bs, Hkv, d, device="cuda")
    k[50, 0, 3] = float("nan")                              # sequence 0
    pkv.paged_kv4_write(k, v, kc, vc, torch.arange(2 * 7 * bs, device="cuda"), bs)
    q = torch.randn(2, Hq, d, device="cuda").bfloat16()
    out = torch.empty_like(q)
    tables = torch.arange(14, dtype=torch.int32, device="cuda").view(2, 7)
    lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode_kv4(out, q, kc, vc, tables, lens, n, 0.1, bs)
    nan = torch.isnan(out).any(-1).cpu()
    assert nan[0, :4].all() and not nan[0, 4:].any() and not nan[1].any()


def test_two_calls_at_once_on_two_streams():
    """Each with its own workspace and output."""
    bs, Hkv, d, Hq, n = 16, 2, 128, 12, 3000
    nb = -(-n // bs)
    kc, vc = (pkv.make_kv4_cache(8 * nb, bs, Hkv, d) for _ in range(2))
    k, v = torch.randn(2, 8 * nb * bs, Hkv, d, device="cuda").bfloat16()
    pkv.paged_kv4_write(k, v, kc, vc, torch.randperm(8 * nb * bs, device="cuda"), bs)
    tables = torch.randperm(8 * nb, device="cuda").int().view(8, nb)
    lens = torch.full((8,), n, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 8, Hq, d, device="cuda").bfloat16()
    ref, got = torch.empty_like(q), torch.empty_like(q)
    ws = [pkv.make_window_workspace(8, Hq, Hkv, d, bs, n, 0) for _ in range(2)]
    for i in range(2):
        pkv.paged_attention_decode_kv4(ref[i], q[i], kc, vc, tables, lens, n, 0.1, bs, workspace=ws[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                pkv.paged_attention_decode_kv4(got[i], q[i], kc, vc, tables, lens, n, 0.1, bs, workspace=ws[i])
    torch.cuda.synchronize()
    assert torch.equal(ref, got)


def test_decode_long_sequence():
    _decode_case(8, 1, 128, 16, [40000, 3], 0, 0, 0)


def test_copied_blocks_decode_alike_and_runs_are_equal():
    """copy_blocks on 4-bit blocks, then the same decode through the copies:
    bit-identical; so are two launches and a captured one."""
    bs, Hkv, d, Hq, n = 16, 2, 128, 12, 700
    nb = -(-n // bs)
    kc, vc = (pkv.make_kv4_cache(2 * nb, bs, Hkv, d) for _ in range(2))
    k, v = torch.randn(2, n, Hkv, d, device="cuda").bfloat16()
    pos = torch.arange(n, device="cuda")
    pkv.paged_kv4_write(k, v, kc, vc, pos, bs)
    pairs = torch.stack([torch.arange(nb), torch.arange(nb) + nb], 1).cuda()
    pkv.copy_blocks([kc], [vc], pairs)
    q = torch.randn(1, Hq, d, device="cuda").bfloat16().repeat(2, 1, 1)
    tables = torch.arange(2 * nb, dtype=torch.int32, device="cuda").view(2, nb)
    lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = pkv.make_window_workspace(2, Hq, Hkv, d, bs, n, 0, 0, 128)
    call = lambda: pkv.paged_attention_decode_kv4(out, q, kc, vc, tables, lens, n, 0.1, bs, partition_size=128,  # noqa: E731
                                                  workspace=ws)
    call()
    first = out.clone()
    assert torch.equal(first[0], first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
