"""The decode of sequences that share blocks, on the GPU against the 64-bit
definition.  Slots that no sequence of the test reads hold NaN, and table
entries past a sequence's blocks are out of range."""
import pytest
import torch

from tests import plain64 as P64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

BF = torch.bfloat16


class Case:
    """groups: (shared tokens, lengths of the members); before, after: lengths of sequences in no group."""

    def __init__(self, groups, Hq, Hkv, d, bs, seed=0, before=(), after=()):
        g = torch.Generator(device="cuda").manual_seed(seed)
        lens, starts, shared, tables = list(before), [], [], []
        need = sum(-(-n // bs) for n in (*before, *after)) + sum(-(-n // bs) for _, ms in groups for n in ms)
        need += sum(-(-P // bs) for P, _ in groups)
        NB = need + 2
        order = (torch.randperm(NB - 1, device="cuda", generator=g) + 1).tolist()

        def take(k):
            return [order.pop() for _ in range(k)]

        tables += [take(-(-n // bs)) for n in before]
        for P, ms in groups:
            starts.append(len(lens))
            shared.append(P)
            head = take(P // bs)
            for n in ms:                                  # a member lists the whole head, however short it is
                tables.append(head + take(max(-(-n // bs) - len(head), 0)))
                lens.append(n)
        starts.append(len(lens))
        lens += list(after)
        tables += [take(-(-n // bs)) for n in after]
        S, MB = len(lens), max(max(len(t) for t in tables), 1)
        tab = torch.full((S, MB), 1 << 30, dtype=torch.int32)
        seen = torch.zeros(NB, bs, dtype=torch.bool)
        for s, t in enumerate(tables):
            tab[s, :len(t)] = torch.tensor(t, dtype=torch.int32)
            for b in range(-(-lens[s] // bs)):
                seen[t[b], :min(bs, lens[s] - b * bs)] = True
        for (P, ms), at in zip(groups, starts):
            for pb in tables[at][:P // bs] if ms else []:
                seen[pb] = True                           # the shared blocks are read whole
        self.kc, self.vc = (torch.randn(NB, bs, Hkv, d, device="cuda", generator=g).to(BF) for _ in range(2))
        for pool in (self.kc, self.vc):
            pool[~seen.cuda()] = float("nan")
        self.q = torch.randn(S, Hq, d, device="cuda", generator=g).to(BF)
        self.tables, self.lens = tab.cuda(), lens
        self.n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.shared = torch.tensor(shared, dtype=torch.int32, device="cuda")
        most = max(shared, default=0)
        self.bounds = (min(max(max(lens), most), MB * bs), min(most, MB * bs),
                       max([len(m) for P, m in groups if P >= bs], default=0))
        self.shape, self.bs, self.scale = (S, Hq, Hkv, d), bs, d ** -0.5

    def run(self, part=0, err_code=0, **kw):
        out = torch.full_like(self.q, 7.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.paged_attention_decode_shared(out, self.q, self.kc, self.vc, self.tables, self.n, self.starts, self.shared,
                                          *self.bounds, self.scale, partition_size=part, err_word=err,
                                          **{"sharing": "always", **kw})
        torch.cuda.synchronize()
        assert int(err) == err_code
        return out

    def check(self, out, absent=()):
        d = self.shape[3]
        for s, n in enumerate(self.lens):
            ids = self.tables[s, :-(-n // self.bs)].long()
            keep = torch.ones(n, dtype=torch.bool, device="cuda")
            for b in range(len(ids)):
                if (s, b) in absent:
                    keep[b * self.bs:(b + 1) * self.bs] = False
            ids = ids.clamp(0, self.kc.shape[0] - 1)
            k, v = (c[ids].flatten(0, 1)[:n] for c in (self.kc, self.vc))
            o, _, mix, reach = P64.attend(self.q[s], k, v, keep, self.scale)
            P64.assert_within(out[s], o, P64.out_bound(o, mix, reach, d, 2.0 ** -8, 2.0 ** -8), f"sequence {s} of {n}")


SHAPES = [(4, 2, 64, 16), (12, 2, 128, 16), (28, 4, 128, 32), (10, 1, 64, 32), (3, 3, 128, 16), (64, 1, 128, 16),
          (200, 1, 64, 16)]
GROUPS = [(304, [305, 344, 304, 400, 320, 999, 306, 310]), (16, [17, 40, 16]), (0, [100, 1, 0]), (1000, [1500, 1001]),
          (128, [129]), (640, [640] * 40), (32, [1200, 33, 50, 64, 65])]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("part", [0, -1, 64, 256])
def test_groups(shape, part):
    c = Case(GROUPS, *shape, seed=1, before=[5, 700], after=[0, 33])
    c.check(c.run(part))


@pytest.mark.parametrize("shape", SHAPES[:3], ids=lambda s: "x".join(map(str, s)))
def test_short_and_empty_members(shape):
    """Members that end inside the shared tokens, and padding of length 0."""
    c = Case([(512, [600, 512, 300, 17, 1, 0, 513]), (256, [0, 0]), (64, [10, 20])], *shape, seed=2)
    for part in (0, 128):
        out = c.run(part)
        c.check(out)
        assert (out[5] == 0).all() and (out[7] == 0).all()


@pytest.mark.parametrize("part", [0, 128])
def test_one_large_group(part):
    """More rows than one unit's tiles, and a prefix over many partitions."""
    c = Case([(2048, [2048 + 3 * i for i in range(75)])], 28, 4, 128, 16, seed=3)
    c.check(c.run(part))


def test_long_document():
    c = Case([(20000, [20001, 20500, 20016]), (9000, [9001, 9100])], 8, 2, 128, 16, seed=4)
    c.check(c.run())


def test_the_choice():
    """auto: a decode without a look at the groups where little is shared, and the shared one where much is."""
    for groups in ([(304, [305, 344, 304, 400])], [(2048, [2050, 3000])], [(304, [1000 + i for i in range(100)])]):
        c = Case(groups, 12, 2, 128, 16, seed=14)
        out = c.run(sharing="auto")
        c.check(out)
        c.starts.fill_(-1)
        assert torch.equal(c.run(sharing="auto"), out)
    c = Case([(4096, [4096 + i for i in range(40)])], 4, 4, 128, 16, seed=15)         # 327 MB read again
    plain = torch.zeros_like(c.q)
    pkv.paged_attention_decode(plain, c.q, c.kc, c.vc, c.tables, c.n, c.bounds[0], c.scale)
    out = c.run(sharing="auto")
    assert torch.equal(out, c.run()) and not torch.equal(out, plain)
    c.check(out)


def test_nothing_shared():
    """Groups that share nothing, or have one member, and no groups at all."""
    for groups in ([(0, [300, 200])], [(208, [300])], [(15, [300, 20])]):
        c = Case(groups, 12, 2, 128, 16, seed=5)
        c.check(c.run())
    c = Case([(64, [100, 200, 300])], 12, 2, 128, 16, seed=6)
    out = torch.zeros_like(c.q)
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode_shared(out, c.q, c.kc, c.vc, c.tables, c.n, empty, empty[:0], 300, 0, 0, c.scale, sharing="always")
    c.check(out)


def test_broken_bounds_are_reported_and_decoded_without_sharing():
    c = Case([(320, [400, 500, 330]), (160, [200, 300])], 12, 2, 128, 16, seed=7)
    good = c.bounds
    c.bounds = (good[0], 300, good[2])                       # shared_lens[0] is above it
    c.check(c.run(err_code=6))
    c.bounds = (good[0], good[1], 2)                         # three members
    c.check(c.run(err_code=6))
    c.bounds = good
    c.shared[1] = -16
    c.check(c.run(err_code=6))
    c.shared[1] = 160
    c.starts[2] = 9                                          # past the last sequence
    c.check(c.run(err_code=6))


@pytest.mark.parametrize("shape", [(12, 2, 128, 16), (4, 2, 64, 32)], ids=lambda s: "x".join(map(str, s)))
def test_bad_blocks_are_absent(shape):
    c = Case([(640, [700, 900, 650]), (128, [300, 400])], *shape, seed=8)
    bs = shape[3]
    absent = set()
    for s, b, bad in [(0, 3, 1 << 20), (1, 3, 1 << 20), (2, 3, 1 << 20), (0, 0, -1), (1, 0, -1), (2, 0, -1),
                      (4, 256 // bs, c.kc.shape[0])]:
        c.tables[s, b] = bad
        absent.add((s, b))
    for part in (0, 128):
        c.check(c.run(part, err_code=1), absent)


def test_growing_logits():
    """Each block's logits exceed the ones before by far more than 2^8: O is rescaled, and the parts' maxima lie apart."""
    c = Case([(1024, [1100, 1500, 1030])], 8, 2, 128, 16, seed=9)
    for s in range(3):
        for b in range(0 if s == 0 else 64, -(-c.lens[s] // 16)):
            pb = int(c.tables[s, b])
            c.kc[pb] = (c.kc[pb].float() * (1 + b / 2)).to(BF)
    for part in (0, 128):
        c.check(c.run(part))


def test_workspaces_graph_and_streams():
    c = Case([(640, [700, 900, 650, 641]), (128, [300, 400])], 12, 2, 128, 16, seed=10)
    S, Hq, Hkv, d = c.shape
    ws = pkv.make_shared_workspace(S, 2, Hq, Hkv, d, 16, *c.bounds, sharing="always")
    want = c.run(workspace=ws)
    c.check(want)
    for _ in range(3):
        assert torch.equal(c.run(workspace=ws), want)
    # smaller workspaces: fewer partitions, or every sequence on its own
    for n in (ws.numel() // 2 // 256 * 256, 70000, 256):
        c.check(c.run(workspace=torch.zeros(n, dtype=torch.uint8, device="cuda")))
    with pytest.raises(pkv.PkvError):
        c.run(part=64, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    out = torch.zeros_like(c.q)

    def step(to=out, space=ws, **kw):
        pkv.paged_attention_decode_shared(to, c.q, c.kc, c.vc, c.tables, c.n, c.starts, c.shared, *c.bounds, c.scale,
                                          workspace=space, sharing="always", **kw)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # other groups in the same graph
    c.shared[0], c.shared[1] = 128, 0
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)
    # two at once, each with a workspace
    others = [torch.zeros_like(out) for _ in range(2)]
    spaces, streams = [ws.clone() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for o, w, st in zip(others, spaces, streams):
            step(o, w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(others[0], out) and torch.equal(others[1], out)


def test_calls_one_behind_the_other():
    """Queued calls of one workspace, whose longest own parts differ, and lengths that the kernel before them writes."""
    cases = [Case([(640, [641, 660]), (32, [40, 50])], 12, 2, 128, 16, seed=12), Case([(64, [3000, 900]), (128, [200, 4000])], 12, 2, 128, 16, seed=13)]
    ws = torch.zeros(max(pkv.shared_workspace_size(4, 2, 12, 2, 128, 16, *c.bounds, 64, "always") for c in cases), dtype=torch.uint8, device="cuda")
    outs = [[torch.zeros_like(c.q) for _ in range(6)] for c in cases]
    kept = [(c.n.clone(), c.starts.clone(), c.shared.clone()) for c in cases]
    torch.cuda.synchronize()
    for i in range(6):
        for c, o, (n, starts, shared) in zip(cases, outs, kept):
            c.n.zero_(), c.starts.zero_(), c.shared.zero_()
            c.n.copy_(n), c.starts.copy_(starts), c.shared.copy_(shared)
            pkv.paged_attention_decode_shared(o[i], c.q, c.kc, c.vc, c.tables, c.n, c.starts, c.shared, *c.bounds, c.scale,
                                              partition_size=64, workspace=ws, sharing="always")
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o[0])
        assert all(torch.equal(x, o[0]) for x in o)


def test_with_the_block_pool():
    """Tables from the host block manager: requests that start with one cached prompt."""
    bs, Hq, Hkv, d = 16, 8, 2, 64
    pool = pkv.BlockPool(200, bs)
    prompt = list(range(1000, 1000 + 100))
    for i in range(6):
        pool.add_sequence(i, prompt + [i] * (5 + 9 * i))
    tabs, lens = pool.block_tables(range(6), 16)
    assert all((tabs[i, :6] == tabs[0, :6]).all() for i in range(6))
    g = torch.Generator(device="cuda").manual_seed(11)
    kc, vc = (torch.randn(200, bs, Hkv, d, device="cuda", generator=g).to(BF) for _ in range(2))
    q = torch.randn(6, Hq, d, device="cuda", generator=g).to(BF)
    t, n = torch.from_numpy(tabs).cuda(), torch.from_numpy(lens).cuda()
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    i32 = dict(dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode(a, q, kc, vc, t, n, int(lens.max()), d ** -0.5)
    pkv.paged_attention_decode_shared(b, q, kc, vc, t, n, torch.tensor([0, 6], **i32), torch.tensor([96], **i32),
                                      int(lens.max()), 96, 6, d ** -0.5)
    for s in range(6):
        k, v = (c[t[s].long()].flatten(0, 1)[:int(lens[s])] for c in (kc, vc))
        o, _, mix, reach = P64.attend(q[s], k, v, torch.ones(int(lens[s]), dtype=torch.bool, device="cuda"), d ** -0.5)
        for x in (a, b):
            P64.assert_within(x[s], o, P64.out_bound(o, mix, reach, d, 2.0 ** -8, 2.0 ** -8), f"sequence {s}")
