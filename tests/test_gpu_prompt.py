"""Attention over whole packed prompts on the GPU against the 64-bit
definition.  The bounds are those of plain64.out_bound: weights rounded to
bf16, logits by their fp32 sums, the output to bf16."""
import pytest
import torch

from tests import plain64 as P64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

BF = torch.bfloat16


def starts(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def seen_by(ql, kl, causal, window, sinks):
    p = kl - ql + torch.arange(ql, device="cuda")[:, None]
    t = torch.arange(kl, device="cuda")[None, :]
    if not causal:
        return torch.ones(ql, kl, dtype=torch.bool, device="cuda")
    ok = t <= p
    if window > 0:
        ok &= (t < sinks) | (t > p - window)
    return ok


def reference(q, k, v, seen, scale):
    """out, mix [ql, Hq, d] and reach [ql, Hq] in 64 bits (plain64.attend, all queries at once)."""
    ql, Hq, d = q.shape
    g = Hq // k.shape[1]
    out = torch.zeros(ql, Hq, d, dtype=torch.float64, device=q.device)
    mix, reach = out.clone(), torch.zeros(ql, Hq, dtype=torch.float64, device=q.device)
    if k.shape[0] == 0:
        return out, mix, reach
    some = seen.any(1)
    for h in range(Hq):
        qh, kh, vh = q[:, h].double(), k[:, h // g].double(), v[:, h // g].double()
        x = (qh @ kh.T * scale).masked_fill(~seen, float("-inf"))
        p = torch.softmax(x, 1)
        p[~some] = 0
        p = p.masked_fill(~seen, 0)
        out[:, h], mix[:, h] = p @ vh, p @ vh.abs()
        reach[:, h] = (qh.abs() @ kh.abs().T * abs(scale)).masked_fill(~seen, 0).amax(1)
    return out, mix, reach


def check(out, q, k, v, ql, kl, causal, window, sinks, scale, what=""):
    d, q0, k0 = q.shape[-1], 0, 0
    for s, (a, b) in enumerate(zip(ql, kl)):
        o, mix, reach = reference(q[q0:q0 + a], k[k0:k0 + b], v[k0:k0 + b], seen_by(a, b, causal, window, sinks), scale)
        bound = P64.out_bound(o.flatten(0, 1), mix.flatten(0, 1), reach.flatten(), d, 2.0 ** -8, 2.0 ** -8)
        P64.assert_within(out[q0:q0 + a].flatten(0, 1), o.flatten(0, 1), bound, f"{what} sequence {s}: {a} queries, {b} keys")
        q0, k0 = q0 + a, k0 + b


def inputs(ql, kl, Hq, Hkv, d, seed=0, packed=False, spare=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if packed:
        rows = torch.randn(sum(ql) + spare, Hq + 2 * Hkv, d, device="cuda", generator=g).to(BF)
        return rows.split([Hq, Hkv, Hkv], 1)
    return [torch.randn(n, h, d, device="cuda", generator=g).to(BF)
            for n, h in ((sum(ql) + spare, Hq), (sum(kl), Hkv), (sum(kl), Hkv))]


def call(q, k, v, ql, kl, causal=True, window=0, sinks=0, scale=None, part=0, **kw):
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    pkv.prompt_attention(out, q, k, v, starts(ql), max(ql), scale, key_start=starts(kl), max_key_len=max(kl), causal=causal,
                         window=window, num_sinks=sinks, partition_size=part, err_word=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out


LENS = [0, 1, 2, 37, 127, 128, 129, 255, 256, 257, 300, 513]
SHAPES = [(4, 2, 64), (12, 2, 128), (28, 4, 128), (10, 1, 64), (3, 3, 128), (5, 5, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both"])
@pytest.mark.parametrize("part", [0, 128, -1])
def test_ragged(shape, causal, part):
    q, k, v = inputs(LENS, LENS, *shape, packed=True)
    out = call(q, k, v, LENS, LENS, causal, part=part)
    check(out, q, k, v, LENS, LENS, causal, 0, 0, shape[2] ** -0.5)


@pytest.mark.parametrize("n", [1, 2, 3, 64, 128, 129, 1000])
@pytest.mark.parametrize("shape", [(1, 1, 64), (7, 1, 128), (12, 2, 128)], ids=lambda s: "x".join(map(str, s)))
def test_one_prompt(n, shape):
    q, k, v = inputs([n], [n], *shape, seed=n)
    for causal in (True, False):
        check(call(q, k, v, [n], [n], causal), q, k, v, [n], [n], causal, 0, 0, shape[2] ** -0.5)


@pytest.mark.parametrize("shape", [(4, 2, 64), (14, 2, 128), (3, 3, 128)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both"])
@pytest.mark.parametrize("part", [0, 128, 384])
def test_queries_and_keys_apart(shape, causal, part):
    """Fewer queries than keys, more (the first ones see nothing), no keys, no queries."""
    ql = [1, 5, 130, 0, 40, 300, 129, 7, 256]
    kl = [700, 129, 1031, 50, 0, 100, 128, 2000, 1]
    q, k, v = inputs(ql, kl, *shape, seed=2)
    out = call(q, k, v, ql, kl, causal, part=part)
    check(out, q, k, v, ql, kl, causal, 0, 0, shape[2] ** -0.5)
    at = sum(ql[:4])
    assert (out[at:at + 40] == 0).all()                               # no keys
    if causal:
        assert (out[at + 40:at + 40 + 200] == 0).all()                # 300 queries, 100 keys
        assert (out[sum(ql[:8]):sum(ql[:8]) + 255] == 0).all()


@pytest.mark.parametrize("shape", [(4, 2, 64), (14, 2, 128), (28, 4, 128)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 130), (128, 0), (257, 3), (1000, 1), (5000, 3),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("part", [0, 128])
def test_window(shape, window, sinks, part):
    ql = [1, 129, 300, 1100, 64, 3]
    kl = [900, 129, 300, 1100, 777, 1]
    q, k, v = inputs(ql, kl, *shape, seed=3)
    out = call(q, k, v, ql, kl, True, window, sinks, part=part)
    check(out, q, k, v, ql, kl, True, window, sinks, shape[2] ** -0.5)


@pytest.mark.parametrize("shape", SHAPES + [(40, 1, 64), (200, 1, 128)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 30, 3), (True, 400, 140)])
@pytest.mark.parametrize("part", [0, 128, 256, -1])
def test_few_queries_each(shape, causal, window, sinks, part):
    """At most 64 queries a sequence: tiles of (query, head) rows, one tile's partitions in pairs."""
    ql = [1, 5, 64, 0, 17, 33, 2, 64, 30, 9]
    kl = [700, 5, 64, 40, 17, 1031, 0, 1500, 29, 4000]
    q, k, v = inputs(ql, kl, *shape, seed=20)
    out = call(q, k, v, ql, kl, causal, window, sinks, part=part)
    check(out, q, k, v, ql, kl, causal, window, sinks, shape[2] ** -0.5)


def test_few_queries_of_a_projection():
    """Rows that hold Q, K and V, and rows whose length is no multiple of a head (then tiles of 128 queries)."""
    ql = [40, 3, 64]
    for width in (12 + 4, 12 + 4.5):
        rows = torch.randn(sum(ql), int(width * 64), device="cuda").to(BF)
        q, k, v = (rows[:, a * 64:b * 64].unflatten(1, (b - a, 64)) for a, b in ((0, 12), (12, 14), (14, 16)))
        check(call(q, k, v, ql, ql), q, k, v, ql, ql, True, 0, 0, 64 ** -0.5)


def test_a_window_over_everything_changes_nothing():
    ql = [400, 129]
    q, k, v = inputs(ql, ql, 12, 2, 128, seed=4)
    assert torch.equal(call(q, k, v, ql, ql), call(q, k, v, ql, ql, window=400))


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0, 1e4])
def test_scales(scale):
    ql = [130, 300]
    q, k, v = inputs(ql, ql, 6, 2, 64, seed=5)
    out = call(q, k, v, ql, ql, scale=scale)
    assert torch.isfinite(out).all()
    if scale < 1e4:                       # beyond, a logit's own fp32 error exceeds what a bound can hold
        check(out, q, k, v, ql, ql, True, 0, 0, scale)


@pytest.mark.parametrize("d,part", [(64, -1), (128, -1), (128, 128)])
def test_growing_logits(d, part):
    """Every stage's largest logit exceeds the earlier ones by more than 2^8, so O is rescaled at each."""
    n = [1300]
    q, k, v = inputs(n, n, 4, 2, d, seed=6)
    k = (k.float() * (1 + torch.arange(n[0], device="cuda") / 20)[:, None, None]).to(BF)
    check(call(q, k, v, n, n, part=part), q, k, v, n, n, True, 0, 0, d ** -0.5)
    check(call(q, k, v, n, n, False, part=part), q, k, v, n, n, False, 0, 0, d ** -0.5)


def test_masked_nan_and_infinities():
    """K values that a query does not see may be anything, and other sequences may hold NaN everywhere."""
    ql = [200, 333, 90]
    q, k, v = inputs(ql, ql, 6, 2, 128, seed=7)
    clean = call(q, k, v, ql, ql)
    for bad in (float("nan"), float("inf"), float("-inf")):
        k2, v2, q2 = k.clone(), v.clone(), q.clone()
        k2[200:533], v2[200:533], q2[200:533] = bad, bad, bad             # the whole middle sequence
        k2[533 + 50] = bad                                                # seen from query 50 of the last one on
        out = call(q2, k2, v2, ql, ql)
        assert torch.equal(out[:200], clean[:200])
        assert torch.equal(out[533:533 + 50], clean[533:533 + 50])
        if bad != bad:
            assert torch.isnan(out[533 + 50:]).all()
        # hidden by a window: keys 60..70 are not seen by queries 180 and on of the first sequence
        k3 = k.clone()
        k3[60:70] = bad
        a, b = call(q, k, v, ql, ql, window=100, sinks=3), call(q, k3, v, ql, ql, window=100, sinks=3)
        assert torch.equal(a[170:200], b[170:200]) and torch.equal(a[:60], b[:60])


def test_rows_behind_the_last_sequence():
    ql = [100, 29]
    q, k, v = inputs(ql, ql, 4, 2, 64, seed=8, spare=300)
    out = call(q, k, v, ql, ql)
    assert (out[129:] == 7.0).all()
    check(out[:129], q[:129], k, v, ql, ql, True, 0, 0, 64 ** -0.5)


def test_bad_starts_are_reported_and_skipped():
    Hq, Hkv, d = 4, 2, 64
    ql = [100, 50, 80]
    q, k, v = inputs(ql, ql, Hq, Hkv, d, seed=9)
    good = call(q, k, v, ql, ql)
    for qs, ks, kept in [([0, 100, 150, 240], [0, 100, 150, 230], [0, 1]),       # past Tq
                         ([0, 100, 90, 230], [0, 100, 150, 230], [0]),           # falling; 140 queries break the bound
                         ([0, 100, 150, 230], [0, 100, 150, 300], [0, 1]),       # past Tk
                         ([-5, 100, 150, 230], [0, 100, 150, 230], [1, 2])]:
        out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.prompt_attention(out, q, k, v, torch.tensor(qs, dtype=torch.int32, device="cuda"), 100, d ** -0.5,
                             key_start=torch.tensor(ks, dtype=torch.int32, device="cuda"), max_key_len=100, err_word=err)
        torch.cuda.synchronize()
        assert int(err) == 6
        for s, (a, b) in enumerate(zip([0, 100, 150], [100, 150, 230])):
            if s in kept:
                assert torch.equal(out[a:b], good[a:b])
        if kept == [0, 1]:
            assert (out[150:] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_over_many_keys(d):
    ql, kl = [3, 1], [20000, 4097]
    q, k, v = inputs(ql, kl, 8, 2, d, seed=10)
    for part in (0, 128, 1024, -1):
        check(call(q, k, v, ql, kl, part=part), q, k, v, ql, kl, True, 0, 0, d ** -0.5, f"partition {part}")
    check(call(q, k, v, ql, kl, window=7000, sinks=5), q, k, v, ql, kl, True, 7000, 5, d ** -0.5)


def test_long_prompt():
    n = [8192]
    q, k, v = inputs(n, n, 4, 1, 128, seed=11)
    check(call(q, k, v, n, n), q, k, v, n, n, True, 0, 0, 128 ** -0.5)


def test_many_sequences():
    """More than one batch of 32 sequences at every level, lengths spread widely."""
    g = torch.Generator().manual_seed(0)
    ql = [int(x) for x in (2 ** (torch.rand(150, generator=g) * 10)).int()]
    q, k, v = inputs(ql, ql, 7, 1, 64, seed=12)
    for part in (0, 128):
        check(call(q, k, v, ql, ql, part=part), q, k, v, ql, ql, True, 0, 0, 64 ** -0.5)


@pytest.mark.parametrize("shape", [(6, 2, 64), (9, 3, 128), (2, 2, 128), (40, 2, 64)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both"])
def test_units_of_one_tile_between_units_of_two(shape, causal):
    # odd numbers of tiles over keys of every length, several units per SM: a tile sits out whole units, and begins
    # its next one while the other tile is still at the one it sat out
    Hq, Hkv, d = shape
    gen = torch.Generator().manual_seed(17)
    ql = [int(torch.randint(1, 129 if i % 3 else 400, (1,), generator=gen)) for i in range(180)]
    kl = [a + int(torch.randint(0, 1500 if i % 2 else 130, (1,), generator=gen)) for i, a in enumerate(ql)]
    if Hq == 40:
        ql = [1 + n % 9 for n in ql]                     # packed: tiles of (query, head) pairs, partitions in pairs
    q, k, v = inputs(ql, kl, Hq, Hkv, d, seed=18)
    part = 256 if Hq == 40 else 0
    out = call(q, k, v, ql, kl, causal, part=part)
    check(out, q, k, v, ql, kl, causal, 0, 0, d ** -0.5)
    for _ in range(20):
        assert torch.equal(call(q, k, v, ql, kl, causal, part=part), out)


def test_repeats_are_equal_and_workspaces_are_reused():
    ql, kl = [3, 100], [5000, 900]
    q, k, v = inputs(ql, kl, 12, 2, 128, seed=13)
    ws = pkv.make_prompt_workspace(2, 103, 100, 5000, 12, 2, 128)
    first = call(q, k, v, ql, kl, workspace=ws)
    for _ in range(3):
        assert torch.equal(call(q, k, v, ql, kl, workspace=ws), first)
    # a smaller one: fewer partitions
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    check(call(q, k, v, ql, kl, workspace=small), q, k, v, ql, kl, True, 0, 0, 128 ** -0.5)
    with pytest.raises(pkv.PkvError):
        call(q, k, v, ql, kl, workspace=small, part=128)


def test_starts_written_by_the_kernel_before():
    ql, kl = [3, 100, 40], [5000, 900, 40]
    q, k, v = inputs(ql, kl, 12, 2, 128, seed=16)
    want = call(q, k, v, ql, kl)
    qs, ks, ws = starts(ql), starts(kl), pkv.make_prompt_workspace(3, 143, 100, 5000, 12, 2, 128)
    a, b = qs.clone(), ks.clone()
    outs = [torch.zeros_like(want) for _ in range(8)]
    torch.cuda.synchronize()
    for o in outs:
        qs.zero_(), ks.zero_()
        qs.copy_(a), ks.copy_(b)
        pkv.prompt_attention(o, q, k, v, qs, 100, 128 ** -0.5, key_start=ks, max_key_len=5000, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_graph_streams_and_two_at_once():
    ql = [300, 200]
    a, b = inputs(ql, ql, 12, 2, 128, seed=14), inputs(ql, ql, 12, 2, 128, seed=15)
    want = [call(*x, ql, ql) for x in (a, b)]
    qs = starts(ql)
    outs = [torch.zeros_like(w) for w in want]
    ws = [pkv.make_prompt_workspace(2, 500, 300, 300, 12, 2, 128) for _ in range(2)]

    def one(i, **kw):
        q, k, v = (a, b)[i]
        pkv.prompt_attention(outs[i], q, k, v, qs, 300, 128 ** -0.5, workspace=ws[i], **kw)

    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            one(i, stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(0)
        one(1)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    # other contents in the same buffers
    for x, y in zip(a, b):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1])
