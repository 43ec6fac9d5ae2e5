"""rotary_kv_write on the GPU.  Its products and sums are rounded to fp32 one
by one and its results once per output, so every output is compared bit for
bit with the same steps taken one at a time on the CPU; the rotation itself is
held against the 64-bit one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

E4M3 = torch.float8_e4m3fn


def table(positions, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat((a.cos(), a.sin()), 1).float()


def rotated(x, cs, rot, interleaved):
    """fp32 on the CPU, an operation at a time."""
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (head[..., ::2], head[..., 1::2]) if interleaved else (head[..., :rot // 2], head[..., rot // 2:])
    ra, rb = a * c - b * s, b * c + a * s
    head = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((head, rest), -1)


def stored(x, dtype, scale):
    if dtype != E4M3:
        return x.to(dtype)
    # the correctly rounded fp32 quotient: 53 bits hold it before its rounding to 24 (53 >= 2 * 24 + 2)
    q = (x.double() / float(torch.tensor(scale, dtype=torch.float32))).float()
    return q.clamp(-448, 448).to(E4M3)


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def case(T, Hq, Hkv, d, rot, bs, dt, cdt, interleaved, packed, seed=0, max_pos=300):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(dt)
    parts = rows.split([Hq, Hkv, Hkv], 1)
    NB = -(-T // bs) + 2
    slots = torch.randperm(NB * bs, generator=g)[:T]
    pos = torch.randint(0, max_pos, (T,), generator=g)
    cs = table(max_pos, rot)
    if T > 3:
        slots[1], pos[2] = -1, -7
    scales = (3.0 / 448, 0.75) if cdt == E4M3 else (1.0, 1.0)
    dev = rows.cuda()
    q, k, v = dev.split([Hq, Hkv, Hkv], 1) if packed else (p.contiguous().cuda() for p in parts)
    pools = [torch.full((NB, bs, Hkv, d), 3.0, device="cuda").to(cdt) for _ in range(2)]
    # what is expected
    live = pos >= 0
    turn = cs[pos.clamp(min=0)]
    rq, rk = (rotated(p, turn, rot, interleaved) for p in parts[:2])
    want_pools = [p.cpu().clone() for p in pools]
    for p, x, sc in zip(want_pools, (rk, parts[2].float()), scales):
        ok = live & (slots >= 0)
        bits(p).view(-1, Hkv, d)[slots[ok]] = bits(stored(x, cdt, sc))[ok]
    return dict(q=q, k=k, v=v, pos=pos.cuda(), cs=cs.cuda(), pools=pools, slots=slots.cuda(), scales=scales, live=live,
                rq=rq.to(dt), rk=rk.to(dt), want=want_pools, parts=parts, turn=turn)


def call(c, q_out, k_out, interleaved, **kw):
    pkv.rotary_kv_write(c["q"], c["k"], c["v"], c["pos"], c["cs"], q_out, k_out, *c["pools"], c["slots"],
                        interleaved=interleaved, k_scale=c["scales"][0], v_scale=c["scales"][1], **kw)


SIZES = [(1, 4, 2, 64, 64, 16), (5, 12, 2, 128, 128, 16), (64, 28, 4, 128, 64, 32), (333, 7, 1, 80, 48, 16),
         (40, 1, 1, 16, 16, 16), (17, 3, 3, 512, 32, 32), (1000, 64, 8, 128, 128, 16), (9, 40, 5, 96, 0, 16)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("cdt", [torch.float32, torch.bfloat16, E4M3], ids=["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("interleaved,packed", [(False, True), (True, False)])
def test_bits(size, dt, cdt, interleaved, packed):
    T, Hq, Hkv, d = size[:4]
    c = case(*size, dt, cdt, interleaved, packed)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((T, Hq, d), 9.0, dtype=dt, device="cuda")
    k_out = torch.full((T, Hkv, d), 9.0, dtype=dt, device="cuda")
    call(c, q_out, k_out, interleaved, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for got, want in ((q_out.cpu(), c["rq"]), (k_out.cpu(), c["rk"])):
        assert torch.equal(bits(got)[c["live"]], bits(want)[c["live"]])
        assert (got[~c["live"]] == 9.0).all()                     # padding tokens are left alone
    for got, want in zip(c["pools"], c["want"]):
        assert torch.equal(bits(got.cpu()), bits(want))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_against_64_bits(interleaved):
    c = case(200, 6, 2, 128, 96, 16, torch.float32, torch.float32, interleaved, False, seed=3)
    q_out = torch.zeros_like(c["q"])
    call(c, q_out, None, interleaved)
    x, half = c["parts"][0].double(), 48
    j = torch.arange(half)
    lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    z = torch.complex(x[..., lo], x[..., hi]) * torch.complex(c["turn"][:, None, :half].double(), c["turn"][:, None, half:].double())
    want, mag = x.clone(), x.abs()
    want[..., lo], want[..., hi] = z.real, z.imag
    size = x[..., lo].abs() + x[..., hi].abs()
    mag[..., lo], mag[..., hi] = size, size
    # two products and a sum, half a step of fp32 each: at most 2 * 2^-24 of |a c| + |b s| <= |a| + |b|
    assert ((q_out.cpu().double() - want).abs()[c["live"]] <= (2 * 2.0 ** -24 * (1 + 2.0 ** -20) * mag)[c["live"]]).all()


def test_in_place_on_a_projection():
    """Q and K rotated where they lie, in rows that hold Q, K and V."""
    T, Hq, Hkv, d = 77, 12, 2, 128
    c = case(T, Hq, Hkv, d, d, 16, torch.bfloat16, torch.bfloat16, False, True, seed=5)
    v = c["v"].clone()
    call(c, c["q"], c["k"], False)
    for got, want in ((c["q"].cpu(), c["rq"]), (c["k"].cpu(), c["rk"])):
        assert torch.equal(got[c["live"]], want[c["live"]])
    assert torch.equal(c["v"], v)
    for got, want in zip(c["pools"], c["want"]):
        assert torch.equal(got.cpu(), want)


def test_without_caches_and_without_queries():
    T, Hq, Hkv, d = 33, 4, 2, 64
    c = case(T, Hq, Hkv, d, 32, 16, torch.bfloat16, torch.bfloat16, True, False, seed=6)
    q_out, k_out = torch.zeros_like(c["q"]), torch.zeros_like(c["k"])
    pkv.rotary_kv_write(c["q"], c["k"], None, c["pos"], c["cs"], q_out, k_out, interleaved=True)
    assert torch.equal(q_out.cpu()[c["live"]], c["rq"][c["live"]]) and torch.equal(k_out.cpu()[c["live"]], c["rk"][c["live"]])
    pkv.rotary_kv_write(None, c["k"], c["v"], c["pos"], c["cs"], None, None, *c["pools"], c["slots"], interleaved=True)
    for got, want in zip(c["pools"], c["want"]):
        assert torch.equal(got.cpu(), want)
    only_q = torch.zeros_like(q_out)
    pkv.rotary_kv_write(c["q"], None, None, c["pos"], c["cs"], only_q, interleaved=True)
    assert torch.equal(only_q, q_out)


def test_bad_positions_and_slots_are_reported():
    T, Hq, Hkv, d = 12, 4, 2, 64
    for which in ("pos", "slot"):
        c = case(T, Hq, Hkv, d, 64, 16, torch.bfloat16, torch.bfloat16, False, False, seed=7)
        pool_before = [p.clone() for p in c["pools"]]
        q_out = torch.full_like(c["q"], 9.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        bad = 5
        if which == "pos":
            c["pos"][bad] = 300
        else:
            c["slots"][bad] = c["pools"][0].shape[0] * 16
        at = int(case(T, Hq, Hkv, d, 64, 16, torch.bfloat16, torch.bfloat16, False, False, seed=7)["slots"][bad])
        call(c, q_out, None, False, err_word=err)
        torch.cuda.synchronize()
        assert int(err) == (8 if which == "pos" else 3)
        # the token's slot keeps what it held; its query is rotated unless its position is the fault
        for got, before in zip(c["pools"], pool_before):
            assert torch.equal(got.view(-1, Hkv, d)[at], before.view(-1, Hkv, d)[at])
        assert bool((q_out[bad] == 9.0).all()) == (which == "pos")
        assert torch.equal(q_out[6].cpu(), c["rq"][6])


def test_non_finite_values_stay_in_their_pair():
    c = case(8, 2, 1, 64, 32, 16, torch.float32, torch.float32, False, False, seed=8)
    c["q"][0, 0, 3] = float("nan")
    c["q"][0, 1, 40] = float("inf")
    q_out = torch.zeros_like(c["q"])
    call(c, q_out, None, False)
    bad = ~torch.isfinite(q_out[0]).cpu()
    assert bad[0].nonzero().flatten().tolist() == [3, 19] and bad[1].nonzero().flatten().tolist() == [40]


def test_graph_and_stream():
    c = case(64, 12, 2, 128, 128, 16, torch.bfloat16, E4M3, False, True, seed=9)
    q_out = torch.zeros(64, 12, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(c, q_out, None, False)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out.cpu()[c["live"]], c["rq"][c["live"]])
    other = torch.cuda.Stream()
    q_out.zero_()
    torch.cuda.synchronize()
    call(c, q_out, None, False, stream=other)
    other.synchronize()
    assert torch.equal(q_out.cpu()[c["live"]], c["rq"][c["live"]])
    for got, want in zip(c["pools"], c["want"]):
        assert torch.equal(bits(got.cpu()), bits(want))


def test_positions_written_by_the_kernel_before():
    c = case(64, 12, 2, 128, 128, 16, torch.bfloat16, torch.bfloat16, False, True, seed=10)
    pos, slots = c["pos"].clone(), c["slots"].clone()
    outs = [torch.zeros(64, 12, 128, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for o in outs:
        c["pos"].zero_(), c["slots"].fill_(-1)
        c["pos"].copy_(pos), c["slots"].copy_(slots)
        call(c, o, None, False)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.cpu()[c["live"]], c["rq"][c["live"]])
    for got, want in zip(c["pools"], c["want"]):
        assert torch.equal(got.cpu(), want)


def test_pool_past_32_bits():
    """Slots whose byte offsets need more than 32 bits."""
    Hkv, d, bs = 8, 128, 32
    NB = (3 << 30) // (bs * Hkv * d) + 1                     # 3 * 2^30 values, 6 GiB a pool
    pools = [torch.zeros(NB, bs, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = (torch.randn(3, Hkv, d, device="cuda").bfloat16() for _ in range(2))
    slots = torch.tensor([NB * bs - 1, 5, NB * bs // 2], device="cuda")
    pos = torch.zeros(3, dtype=torch.int64, device="cuda")
    pkv.rotary_kv_write(None, k, v, pos, table(1, 128).cuda(), None, None, *pools, slots)
    for p, x in zip(pools, (k, v)):
        assert torch.equal(p.view(-1, Hkv, d)[slots], x)      # position 0 turns nothing
