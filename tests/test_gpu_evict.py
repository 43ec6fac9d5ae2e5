"""Eviction by accumulated attention weight on the GPU: the scored decode
against 64 bits, the choice of tokens against a sort, and a whole cycle of
scored decode, eviction, repacking and decode."""
import math

import numpy as np
import pytest
import torch

from tests import plain64 as P64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

E4M3 = torch.float8_e4m3fn


def _pools(NB, bs, Hkv, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    sc = 5.0 / 448 if dtype == E4M3 else 1.0
    k, v = ((torch.randn(NB, bs, Hkv, d, device="cuda", generator=g) / sc).clamp(-448, 448).to(dtype) for _ in range(2))
    return k, v, sc


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d,bs", [(12, 2, 128, 16), (7, 1, 64, 32), (10, 1, 128, 16), (3, 3, 64, 16),
                                         (64, 8, 128, 32)])
@pytest.mark.parametrize("part", [0, -1, 128])
def test_scored_decode(dtype, Hq, Hkv, d, bs, part):
    lens = [0, 1, 31, 32, 33, 500, 2000]
    S, MT = len(lens), max(lens) + 5
    NB = -(-S * MT // bs)
    k, v, sc = _pools(NB, bs, Hkv, d, dtype, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    slots = torch.randperm(NB * bs, device="cuda", generator=g)[:S * MT].view(S, MT).int()
    slots[4, 7] = NB * bs                                  # absent: weight 0
    q = torch.randn(S, Hq, d, device="cuda", generator=g).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = torch.rand(S, MT, device="cuda", generator=g)
    scores, err = before.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pkv.make_scored_workspace(S, Hq, Hkv, d, bs, max(lens), part)
    out, plain = torch.empty_like(q), torch.empty_like(q)
    kw = dict(scale=d ** -0.5, k_scale=sc, v_scale=sc, partition_size=part)
    pkv.token_attention_decode_scored(out, q, k, v, slots, n, scores, max(lens), workspace=ws, err_word=err, **kw)
    pkv.token_attention_decode(plain, q, k, v, slots, n, max(lens), **kw)
    assert int(err) == 3
    if part != 0:                                          # the library's own choice may split further
        assert torch.equal(out, plain)
    again = before.clone()
    pkv.token_attention_decode_scored(out, q, k, v, slots, n, again, max(lens), workspace=ws, **kw)
    assert torch.equal(again, scores)
    flat = [c.flatten(0, 1) for c in (k, v)]
    for s, m in enumerate(lens):
        assert torch.equal(scores[s, m:], before[s, m:])
        ok = slots[s, :m] < NB * bs
        idx = torch.where(ok, slots[s, :m], 0).long()
        o, w, mix, reach = P64.attend(q[s], flat[0][idx].double() * sc, flat[1][idx].double() * sc, ok, d ** -0.5)
        p_eps, small = (2.0 ** -8, 0.0) if dtype == torch.bfloat16 else (2.0 ** -11, m * 2.0 ** -25 * 6.0)
        P64.assert_within(out[s], o, P64.out_bound(o, mix, reach, d, p_eps, 2.0 ** -8, small), f"output of {m}")
        # a weight is off by the logits' error on both sides of the division and a few roundings;
        # the sum by a rounding per head
        rel = 2 * P64.logit_slack(reach, d)[:, None] + 2.0 ** -19 + Hq * 2.0 ** -24
        want = before[s, :m].double() + w.sum(0)
        P64.assert_within(scores[s, :m], want, (rel * w).sum(0) + 2.0 ** -24 * want + 1e-30, f"scores of {m}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d,bs", [(12, 2, 128, 16), (7, 1, 64, 32)])
def test_tables_whose_slots_follow_one_another(dtype, Hq, Hkv, d, bs):
    """Runs of 16 and more, from the pool's first slot, at odd slots across blocks, up to its last slot, broken by one
    slot, by an absent one or in falling order: the same bits as the same rows scattered over another pool."""
    NB, MT = 40, 640
    P = NB * bs
    k, v, sc = _pools(NB, bs, Hkv, d, dtype, 11)
    up = lambda a, m: list(range(a, a + m))  # noqa: E731
    rows = [up(0, 640), up(P - 640, 640), up(7, 331), up(0, 16) + up(64, 16) + up(1, 48) + up(P - 33, 33),
            up(0, 40) + [90] + up(41, 200), up(0, 100) + [P + 3] + up(101, 100), up(32, 64)[::-1] + up(0, 64),
            up(48, 8) + up(48, 8) + up(48, 16), up(5, 16), up(5, 15), []]
    S = len(rows)
    slots = torch.full((S, MT), -5, dtype=torch.int32)
    for s, row in enumerate(rows):
        slots[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
    slots = slots.cuda()
    n = torch.tensor([len(r) for r in rows], dtype=torch.int32, device="cuda")
    move = torch.randperm(P, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    assert int((move[1:] == move[:-1] + 1).sum()) < 16
    k2, v2 = (torch.empty_like(c) for c in (k, v))
    k2.flatten(0, 1)[move], v2.flatten(0, 1)[move] = k.flatten(0, 1), v.flatten(0, 1)
    live = (slots >= 0) & (slots < P)
    slots2 = torch.where(live, move[torch.where(live, slots, 0).long()].int(), slots)
    q = torch.randn(S, Hq, d, device="cuda").bfloat16()
    kw = dict(scale=d ** -0.5, k_scale=sc, v_scale=sc, partition_size=128)
    got = []
    for kc, vc, tab in ((k, v, slots), (k2, v2, slots2)):
        out, scored, weights = torch.empty_like(q), torch.empty_like(q), torch.zeros(S, MT, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.token_attention_decode(out, q, kc, vc, tab, n, MT, err_word=err, **kw)
        pkv.token_attention_decode_scored(scored, q, kc, vc, tab, n, weights, MT, **kw)
        assert int(err) == 3 and torch.equal(out, scored)
        got.append((out, weights))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    p_eps, small = (2.0 ** -8, 0.0) if dtype == torch.bfloat16 else (2.0 ** -11, MT * 2.0 ** -25 * 6.0)
    for s, row in enumerate(rows):
        ok = live[s, :len(row)]
        idx = torch.where(ok, slots[s, :len(row)], 0).long()
        o, w, mix, reach = P64.attend(q[s], k.flatten(0, 1)[idx].double() * sc, v.flatten(0, 1)[idx].double() * sc, ok,
                                      d ** -0.5)
        P64.assert_within(got[0][0][s], o, P64.out_bound(o, mix, reach, d, p_eps, 2.0 ** -8, small), f"row {s}")


def _evict_reference(slots, scores, n, budget, first, recent):
    if n <= budget:
        keep = list(range(n))
    else:
        rest = sorted(range(first, n - recent), key=lambda i: (-(scores[i] if scores[i] == scores[i] else -math.inf),
                                                               scores[i] != scores[i], i))
        keep = sorted(list(range(first)) + rest[:budget - first - recent] + list(range(n - recent, n)))
    gone = sorted(set(range(n)) - set(keep))
    return [slots[i] for i in keep], [scores[i] for i in keep], [slots[i] for i in gone]


def _scores(kind, S, MT, rng):
    x = rng.random((S, MT)).astype(np.float32) ** 4
    if kind == "ties":
        x = np.round(x * 3).astype(np.float32)
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "wild":
        x = rng.standard_normal((S, MT)).astype(np.float32) * np.float32(10) ** rng.integers(-38, 38, (S, MT))
        for val in (np.nan, np.inf, -np.inf, 0.0, -0.0, -np.nan, 1e-45):
            x[rng.random((S, MT)) < 0.05] = val
    return x.astype(np.float32)


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "wild"])
@pytest.mark.parametrize("lens,budget,first,recent", [
    ([0, 1, 5, 8, 9, 100], 8, 2, 3), ([1023, 1024, 1025, 4097, 700], 700, 4, 128), ([3000, 50], 0, 0, 0),
    ([3000, 2999, 3001], 3000, 1500, 1500), ([5000], 1, 0, 0), ([20000, 16385, 9000], 8192, 0, 1),
    ([70001, 131072, 262143], 33333, 16, 2000), ([500, 400], 300, 300, 0), ([500, 400], 300, 0, 300)])
def test_evict(kind, lens, budget, first, recent):
    S, MT = len(lens), max(lens) + 3
    rng = np.random.default_rng(len(lens) + budget)
    scores = _scores(kind, S, MT, rng)
    slots = rng.permutation(S * MT).reshape(S, MT).astype(np.int32)
    ns, nsc = torch.full((S, MT), -9, dtype=torch.int32, device="cuda"), torch.full((S, MT), -9.0, device="cuda")
    nn, ev = torch.full((S,), -9, dtype=torch.int32, device="cuda"), torch.full((S, MT), -9, dtype=torch.int32, device="cuda")
    pkv.evict_tokens(torch.from_numpy(slots).cuda(), torch.from_numpy(scores).cuda(),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), ns, nsc, nn, budget, first, recent, ev)
    ns, nsc, nn, ev = (x.cpu().numpy() for x in (ns, nsc, nn, ev))
    for s, n in enumerate(lens):
        a, b, c = _evict_reference(slots[s].tolist(), scores[s].tolist(), n, budget, first, recent)
        assert nn[s] == len(a)
        assert ns[s].tolist() == a + [-9] * (MT - len(a))
        np.testing.assert_array_equal(nsc[s][:len(b)], np.array(b, np.float32))
        assert (nsc[s][len(b):] == -9).all()
        assert ev[s].tolist() == c + [-9] * (MT - len(c))


def test_evict_in_a_graph_over_a_cluster():
    """A few long sequences (several blocks each), captured and replayed on other scores and counts, on two streams."""
    S, MT = 2, 40000
    rng = np.random.default_rng(7)
    slots = torch.from_numpy(rng.permutation(S * MT).reshape(S, MT).astype(np.int32)).cuda()
    scores, n = torch.zeros(S, MT, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    ns, nsc, nn, ev = torch.zeros_like(slots), torch.zeros_like(scores), torch.zeros_like(n), torch.zeros_like(slots)
    call = lambda: pkv.evict_tokens(slots, scores, n, ns, nsc, nn, 5000, 4, 100, ev)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed, lens in ((1, [40000, 5001]), (2, [5000, 33333])):
        x = _scores("ties", S, MT, np.random.default_rng(seed))
        scores.copy_(torch.from_numpy(x))
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        other = [torch.zeros_like(t) for t in (ns, nsc, nn)]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            pkv.evict_tokens(slots, scores, n, *other, 5000, 4, 100)
        graph.replay()
        torch.cuda.synchronize()
        for s, m in enumerate(lens):
            a, b, c = _evict_reference(slots[s].tolist(), x[s].tolist(), m, 5000, 4, 100)
            assert ns[s, :len(a)].tolist() == a and ev[s, :len(c)].tolist() == c and int(nn[s]) == len(a)
            assert other[0][s, :len(a)].tolist() == a
            np.testing.assert_array_equal(nsc[s, :len(b)].cpu().numpy(), np.array(b, np.float32))


@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_scored_decode_with_other_logit_scales(scale):
    S, MT, Hq, Hkv, d, bs = 2, 700, 6, 2, 64, 16
    k, v, _ = _pools(100, bs, Hkv, d, torch.bfloat16, 3)
    slots = torch.randperm(1600, device="cuda")[:S * MT].view(S, MT).int()
    q = torch.randn(S, Hq, d, device="cuda").bfloat16()
    n, scores = torch.tensor([700, 13], dtype=torch.int32, device="cuda"), torch.zeros(S, MT, device="cuda")
    pkv.token_attention_decode_scored(torch.empty_like(q), q, k, v, slots, n, scores, MT, scale, partition_size=128)
    for s, m in enumerate((700, 13)):
        idx = slots[s, :m].long()
        _, w, _, reach = P64.attend(q[s], k.flatten(0, 1)[idx], v.flatten(0, 1)[idx],
                                    torch.ones(m, dtype=torch.bool, device="cuda"), scale)
        P64.assert_within(scores[s, :m], w.sum(0), ((2 * P64.logit_slack(reach, d)[:, None] + 2.0 ** -18) * w).sum(0))


def test_evict_without_a_list_and_with_bad_counts():
    S, MT = 3, 300
    rng = np.random.default_rng(1)
    scores, slots = _scores("plain", S, MT, rng), rng.permutation(S * MT).reshape(S, MT).astype(np.int32)
    ns, nsc = torch.zeros((S, MT), dtype=torch.int32, device="cuda"), torch.zeros((S, MT), device="cuda")
    nn, err = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    n = torch.tensor([-4, 301, 200], dtype=torch.int32, device="cuda")
    pkv.evict_tokens(torch.from_numpy(slots).cuda(), torch.from_numpy(scores).cuda(), n, ns, nsc, nn, 100, 4, 10,
                     err_word=err)
    assert int(err) == 2
    assert nn.tolist() == [0, 100, 100]
    for s, m in ((1, 300), (2, 200)):
        a, _, _ = _evict_reference(slots[s].tolist(), scores[s].tolist(), m, 100, 4, 10)
        assert ns[s, :100].tolist() == a


def test_cycle_of_scored_decode_eviction_repacking_and_decode():
    """A few scored steps, eviction to a budget, repacking of the survivors'
    blocks, and a decode over what is left: it equals the decode before the
    repack bit for bit and the 64-bit attention over the kept tokens."""
    bs, Hq, Hkv, d = 16, 12, 2, 128
    lens = [700, 90, 1300]
    MT = 1400
    NB = sum(-(-m // bs) for m in lens) + 1
    k, v, _ = _pools(NB, bs, Hkv, d, torch.bfloat16, 8)
    ids, at = np.random.default_rng(2).permutation(NB - 1) + 1, 0
    slots = np.zeros((3, MT), np.int32)
    for s, m in enumerate(lens):
        t = np.arange(m)
        slots[s, :m] = ids[at + t // bs] * bs + t % bs
        at += -(-m // bs)
    tab = torch.from_numpy(slots).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scores = torch.zeros(3, MT, device="cuda")
    ws = pkv.make_scored_workspace(3, Hq, Hkv, d, bs, max(lens))
    total = torch.zeros(3, MT, dtype=torch.float64, device="cuda")
    for step in range(3):
        q = torch.randn(3, Hq, d, device="cuda").bfloat16() * 2
        out = torch.empty_like(q)
        pkv.token_attention_decode_scored(out, q, k, v, tab, n, scores, max(lens), d ** -0.5, workspace=ws)
        for s, m in enumerate(lens):
            idx = tab[s, :m].long()
            total[s, :m] += P64.attend(q[s], k.flatten(0, 1)[idx], v.flatten(0, 1)[idx],
                                       torch.ones(m, dtype=torch.bool, device="cuda"), d ** -0.5)[1].sum(0)
    assert torch.allclose(scores.double(), total, rtol=1e-4, atol=1e-7)
    new, nscore = torch.zeros_like(tab), torch.zeros_like(scores)
    nn, gone = torch.zeros_like(n), torch.zeros_like(tab)
    pkv.evict_tokens(tab, scores, n, new, nscore, nn, 200, 4, 64, gone)
    kept = nn.tolist()
    assert kept == [200, 90, 200]
    for s, m in enumerate(lens):
        assert sorted(new[s, :kept[s]].tolist() + gone[s, :m - kept[s]].tolist()) == sorted(slots[s, :m].tolist())
    q = torch.randn(3, Hq, d, device="cuda").bfloat16()
    a, b = torch.empty_like(q), torch.empty_like(q)
    pkv.token_attention_decode(a, q, k, v, new, nn, 200, d ** -0.5)
    for s in range(3):
        idx = new[s, :kept[s]].long()
        o, _, mix, reach = P64.attend(q[s], k.flatten(0, 1)[idx], v.flatten(0, 1)[idx],
                                      torch.ones(kept[s], dtype=torch.bool, device="cuda"), d ** -0.5)
        P64.assert_within(a[s], o, P64.out_bound(o, mix, reach, d, 2.0 ** -8, 2.0 ** -8))
    moves, freed = pkv.vtoken_plan(new.cpu().numpy(), nn.cpu().numpy(), bs, NB)
    assert len(moves) and len(freed)
    pkv.repack_tokens([k], [v], new, torch.from_numpy(moves).cuda())
    k[torch.from_numpy(freed).long().cuda()] = float("nan")
    v[torch.from_numpy(freed).long().cuda()] = float("nan")
    pkv.token_attention_decode(b, q, k, v, new, nn, 200, d ** -0.5)
    assert torch.equal(a, b)


def test_two_captured_steps_share_nothing_but_the_workspace():
    """Scored decode and eviction captured together and replayed twice."""
    S, MT, bs, Hq, Hkv, d = 4, 900, 16, 8, 2, 64
    NB = S * MT // bs + 1
    k, v, _ = _pools(NB, bs, Hkv, d, torch.bfloat16, 5)
    slots = torch.randperm(NB * bs, device="cuda")[:S * MT].view(S, MT).int()
    n = torch.tensor([900, 1, 450, 899], dtype=torch.int32, device="cuda")
    q = torch.randn(S, Hq, d, device="cuda").bfloat16()
    out, scores = torch.empty_like(q), torch.zeros(S, MT, device="cuda")
    ns, nsc, nn = torch.zeros_like(slots), torch.zeros_like(scores), torch.zeros_like(n)
    ws = pkv.make_scored_workspace(S, Hq, Hkv, d, bs, MT, 128)

    def step():
        pkv.token_attention_decode_scored(out, q, k, v, slots, n, scores, MT, 0.125, partition_size=128, workspace=ws)
        pkv.evict_tokens(slots, scores, n, ns, nsc, nn, 300, 4, 32)

    step()
    eager = [x.clone() for x in (out, scores, ns, nsc, nn)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        scores.zero_()
        ns.zero_()
        nsc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((out, scores, ns, nsc, nn), eager):
            assert torch.equal(x, y)
