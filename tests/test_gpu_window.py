"""Attention under a sliding window with sinks, decode and query chunks, on
the GPU against the 64-bit definition.  Everything a call must not read is
poisoned: hidden tokens hold NaN, and table entries of blocks no query sees
are out of range (they would be reported)."""
import numpy as np
import pytest
import torch

from tests import plain64 as P64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

E4M3 = torch.float8_e4m3fn


def _pool(lens, Hkv, d, bs, dtype, seed, seen_of):
    """Shuffled pool with NaN in every slot no query sees, the tables with
    entries out of range for unseen blocks, and dense K/V per sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nblk = [-(-n // bs) for n in lens]
    NB = sum(nblk) + 2
    order = (torch.randperm(NB - 1, device="cuda", generator=g) + 1).tolist()
    MB = max(max(nblk), 1)
    tables = torch.full((len(lens), MB), 1 << 30, dtype=torch.int32)
    pools, dense, scale = [], [[], []], 1.0
    if dtype == E4M3:
        scale = 5.0 / 448
    for side in range(2):
        x = torch.randn(NB, bs, Hkv, d, device="cuda", generator=g)
        pools.append((x / scale).clamp(-448, 448).to(dtype))
    at = 0
    hide = torch.ones(NB, bs, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        ids = order[at:at + nblk[s]]
        at += nblk[s]
        seen = seen_of(s, n)
        for b, pb in enumerate(ids):
            live = seen[b * bs:(b + 1) * bs]
            if live.any():
                tables[s, b] = pb
            hide[pb, :live.numel()] = ~live
        idx = torch.tensor(ids, dtype=torch.long, device="cuda")
        for side in range(2):
            dense[side].append(pools[side][idx].double().flatten(0, 1)[:n] * scale)
    for p in pools:
        if dtype == E4M3:
            p.view(torch.uint8)[hide] = 0x7F
        else:
            p[hide] = float("nan")
    return pools, tables.cuda(), dense, scale


def _decode_case(dtype, Hq, Hkv, d, bs, lens, window, sinks, part, kernel, seed=1, scale=None):
    seen_of = lambda s, n: P64.window_seen(n, n - 1, window, sinks)  # noqa: E731
    (kc, vc), tables, dense, sc = _pool(lens, Hkv, d, bs, dtype, seed, seen_of)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    qdt = torch.float32 if dtype == torch.float32 else torch.bfloat16
    q = torch.randn(len(lens), Hq, d, device="cuda", generator=g).to(qdt)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx, scale = max(lens), d ** -0.5 if scale is None else scale
    ws = pkv.make_window_workspace(len(lens), Hq, Hkv, d, bs, mx, window, sinks, part)
    pkv.paged_attention_decode_window(out, q, kc, vc, tables, n, mx, scale, window, sinks, k_scale=sc, v_scale=sc,
                                      partition_size=part, workspace=ws, err_word=err, kernel=kernel)
    torch.cuda.synchronize()
    assert int(err) == 0
    # the tensor-core kernel rounds the weights: to bf16 with a bf16 cache, to fp16 with E4M3
    tc = kernel != "cuda_cores" and dtype != torch.float32
    p_eps = (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11) if tc else 0.0
    for s, m in enumerate(lens):
        k, v = dense[0][s], dense[1][s]
        o, _, mix, reach = P64.attend(q[s], k, v, seen_of(s, m), scale)
        small = m * 2.0 ** -25 * float(v.abs().max()) if tc and dtype == E4M3 and m else 0.0   # fp16 weights below 2^-14
        P64.assert_within(out[s], o, P64.out_bound(o, mix, reach, d, p_eps, P64.HALF[qdt], small),
                          f"sequence {s} of {m} tokens")
    return out


LENS = [0, 1, 15, 16, 17, 37, 300, 1000, 2049]
SHAPES = [(4, 2, 64, 16), (12, 2, 128, 16), (28, 4, 128, 32), (10, 1, 64, 32), (3, 3, 128, 16)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, E4M3], ids=["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (17, 33), (100, 1), (999, 16), (5000, 3), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode(dtype, shape, window, sinks):
    _decode_case(dtype, *shape, LENS, window, sinks, 0, "auto")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, E4M3], ids=["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("part", [-1, 16, 32, 48, 64, 128])
@pytest.mark.parametrize("kernel", ["auto", "cuda_cores"])
def test_decode_partitions(dtype, part, kernel):
    _decode_case(dtype, 16, 2, 128, 16, LENS, 777, 20, part, kernel)
    _decode_case(dtype, 8, 2, 64, 32, [5000, 1, 700], 1300, 70, part if part % 32 == 0 else -1, kernel)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, E4M3], ids=["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 2.0])
def test_decode_with_other_logit_scales(dtype, scale):
    _decode_case(dtype, 12, 2, 128, 16, [1, 100, 1500], 900, 3, 128, "auto", scale=scale)
    _decode_case(dtype, 7, 1, 64, 32, [33, 700], 100, 5, 0, "auto", scale=scale)


def test_fp32_offsets_past_32_bits():
    """An fp32 pool of more than 2^32 bytes, the sequence in its last blocks."""
    bs, Hkv, d, Hq, n = 16, 8, 128, 16, 300
    NB = (1 << 32) // (bs * Hkv * d * 4) + 100
    kc, vc = torch.zeros(2, NB, bs, Hkv, d, device="cuda")
    ids = NB - 1 - torch.arange(-(-n // bs), device="cuda")
    for c in (kc, vc):
        c[ids] = torch.randn(ids.numel(), bs, Hkv, d, device="cuda")
    q = torch.randn(1, Hq, d, device="cuda")
    for kernel in ("auto", "cuda_cores"):
        out = torch.empty_like(q)
        pkv.paged_attention_decode_window(out, q, kc, vc, ids.int()[None].contiguous(),
                                          torch.tensor([n], dtype=torch.int32, device="cuda"), n, 0.1, 200, 4,
                                          kernel=kernel)
        o, _, mix, reach = P64.attend(q[0], kc[ids].flatten(0, 1)[:n], vc[ids].flatten(0, 1)[:n],
                                      P64.window_seen(n, n - 1, 200, 4), 0.1)
        P64.assert_within(out[0], o, P64.out_bound(o, mix, reach, d, 0.0, 2.0 ** -24), kernel)


def test_bf16_query_over_an_fp32_cache():
    """The one mix of dtypes the tensor cores do not take."""
    lens = [1, 40, 700]
    seen_of = lambda s, n: P64.window_seen(n, n - 1, 300, 2)  # noqa: E731
    (kc, vc), tables, dense, _ = _pool(lens, 2, 128, 16, torch.float32, 5, seen_of)
    q = torch.randn(3, 12, 128, device="cuda").bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for kernel in ("auto", "cuda_cores"):
        out = torch.empty_like(q)
        pkv.paged_attention_decode_window(out, q, kc, vc, tables, n, 700, 0.1, 300, 2, kernel=kernel)
        for s, m in enumerate(lens):
            o, _, mix, reach = P64.attend(q[s], dense[0][s], dense[1][s], seen_of(s, m), 0.1)
            P64.assert_within(out[s], o, P64.out_bound(o, mix, reach, 128, 0.0, 2.0 ** -8), f"{kernel} {m}")


def test_window_of_every_token_equals_the_plain_decode():
    for dtype, kernel in ((torch.bfloat16, "auto"), (torch.bfloat16, "cuda_cores"), (torch.float32, "cuda_cores")):
        lens = [1, 40, 700, 1500]
        (kc, vc), tables, _, _ = _pool(lens, 2, 128, 16, dtype, 5, lambda s, n: P64.window_seen(n, n, 0, 0))
        q = torch.randn(4, 12, 128, device="cuda").to(dtype)
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        a, b = torch.empty_like(q), torch.empty_like(q)
        pkv.paged_attention_decode(a, q, kc, vc, tables, n, 1500, 0.1, partition_size=128, kernel=kernel)
        pkv.paged_attention_decode_window(b, q, kc, vc, tables, n, 1500, 0.1, 1500, 0, partition_size=128, kernel=kernel)
        assert torch.equal(a, b)


def _prefill_case(Hq, Hkv, d, bs, chunks, window, sinks, part, seed=3, scale=None):
    """chunks: (queries, length) per sequence."""
    def seen_of(s, n):
        ql = chunks[s][0]
        ok = torch.zeros(n, dtype=torch.bool, device="cuda")
        for i in range(ql):
            ok |= P64.window_seen(n, n - ql + i, window, sinks)
        return ok
    lens = [n for _, n in chunks]
    (kc, vc), tables, dense, _ = _pool(lens, Hkv, d, bs, torch.bfloat16, seed, seen_of)
    T = sum(c[0] for c in chunks)
    q = torch.randn(T, Hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16()
    start = torch.tensor(np.concatenate([[0], np.cumsum([c[0] for c in chunks])]), dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mq, mx = max(c[0] for c in chunks), max(lens)
    ws = pkv.make_prefill_window_workspace(len(chunks), T, mq, Hq, Hkv, d, bs, mx, window, sinks, part)
    scale = d ** -0.5 if scale is None else scale
    pkv.paged_attention_prefill_window(out, q, kc, vc, tables, n, start, mq, mx, scale, window, sinks,
                                       partition_size=part, workspace=ws, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    at = 0
    for s, (ql, m) in enumerate(chunks):
        rows = range(ql) if ql <= 40 else sorted({0, 1, ql // 3, ql // 2, ql - 2, ql - 1, 18 % ql, 37 % ql})
        for i in rows:
            o, _, mix, reach = P64.attend(q[at + i], dense[0][s], dense[1][s],
                                          P64.window_seen(m, m - ql + i, window, sinks), scale)
            P64.assert_within(out[at + i], o, P64.out_bound(o, mix, reach, d, 2.0 ** -8, 2.0 ** -8),
                              f"query {i} of {ql}, length {m}")
        at += ql


CHUNKS = [(1, 1), (5, 5), (0, 9), (17, 40), (100, 300), (130, 1000), (257, 2050), (1, 1999)]


@pytest.mark.parametrize("shape", [(12, 2, 128, 16), (8, 8, 64, 32), (28, 4, 128, 16), (10, 1, 64, 16)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (64, 40), (300, 0), (300, 5), (4096, 4)])
@pytest.mark.parametrize("part", [0, -1, 64])
def test_prefill(shape, window, sinks, part):
    _prefill_case(*shape, CHUNKS, window, sinks, part)


def test_prefill_few_queries_takes_the_single_tile_kernel():
    _prefill_case(28, 4, 128, 16, [(5, 3000), (5, 5), (2, 1200)], 1000, 4, 0)


@pytest.mark.parametrize("g", [1, 2, 3, 5, 6, 9, 12, 28, 48, 100, 128, 130])
def test_prefill_group_sizes(g):
    """Tiles that begin and end inside a query, hold one query, or less than one."""
    ql = max(4, 600 // g)
    _prefill_case(g, 1, 128, 16, [(ql, ql + 100), (ql // 2, ql // 2), (3, 400)], 130, 3, 0)
    _prefill_case(2 * g, 2, 64, 32, [(ql, ql)], 64, 0, 0)


@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_prefill_with_other_logit_scales(scale):
    _prefill_case(14, 2, 128, 16, [(200, 700), (1, 50)], 150, 4, 0, scale=scale)


def test_bad_block_and_length_are_reported():
    lens = [100, 300]
    (kc, vc), tables, dense, _ = _pool(lens, 2, 128, 16, torch.bfloat16, 9, lambda s, n: P64.window_seen(n, n - 1, 64, 4))
    tables[0, 5] = -3                                      # inside the first sequence's window
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, err = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode_window(out, q, kc, vc, tables, n, 300, 0.1, 64, 4, err_word=err)
    assert int(err) == 1
    seen = P64.window_seen(100, 99, 64, 4)
    seen[80:96] = False                                    # the block is skipped, the others are attended
    for s, ok in ((0, seen), (1, P64.window_seen(300, 299, 64, 4))):
        o, _, mix, reach = P64.attend(q[s], dense[0][s], dense[1][s], ok, 0.1)
        P64.assert_within(out[s], o, P64.out_bound(o, mix, reach, 128, 2.0 ** -8, 2.0 ** -8))
    (kc, vc), tables, _, _ = _pool(lens, 2, 128, 16, torch.bfloat16, 9, lambda s, n: P64.window_seen(n, n, 0, 0))
    err.zero_()
    pkv.paged_attention_decode_window(out, q, kc, vc, tables, n, 128, 0.1, 64, 4, err_word=err)
    assert int(err) == 2


def test_stream_and_graph():
    """On a side stream, captured into a graph and replayed with new lengths."""
    lens = [200, 1500, 33]
    (kc, vc), tables, dense, _ = _pool(lens, 2, 128, 16, torch.bfloat16, 11, lambda s, n: P64.window_seen(n, n, 0, 0))
    q = torch.randn(3, 12, 128, device="cuda").bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = pkv.make_window_workspace(3, 12, 2, 128, 16, 1500, 700, 4, 128)
    call = lambda: pkv.paged_attention_decode_window(out, q, kc, vc, tables, n, 1500, 0.1, 700, 4,  # noqa: E731
                                                     partition_size=128, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    n.copy_(torch.tensor([150, 1400, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    call()
    assert torch.equal(out, replayed) and not torch.equal(first, replayed)
