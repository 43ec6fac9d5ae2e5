"""The 4-bit decode against 64 bits with bounds made of the actual weights,
scales and codes: values of every size, long sequences, few and many heavy
tokens.  The bound of a case is tight enough to refuse an output of zeros and
one that leaves out a stage or a partition (planted in the 64-bit form)."""
import pytest
import torch

from tests import plain64 as P64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

STAGE = 64             # tokens of a stage


def _weights(q, k, scale, seen):
    x = (k.double() @ q.double()) * scale
    return torch.softmax(x.masked_fill(~seen, float("-inf")), 0)


def reference(q, k, v, seen, scale, v_scale, unit):
    """q [Hq, d], k/v [n, Hkv, d] (the values the cache stands for): the
    64-bit output [Hq, d] and a bound on the kernel's distance from it.

    With p the weights (largest 1), the kernel sums z p' and c fp16(s p') in
    fp32, p' = fp16(p): p' is off by 2^-11 relative, and by the logit's error
    on either side of the division, which moves the mean by that times
    sum w |v - o|; fp16(s p') is off by 2^-11, times sum w |s c|; the sums by
    two units of 2^-23 of the magnitudes per 16 tokens of a unit; the output
    by bf16's half step.  The weights carry 2^12, so what is below fp16's
    smallest normal number is off by 2^-25 / 2^12 per token (and by the power
    of two that a scale of 2 or more takes off again)."""
    q, k, v = q.double(), k.double(), v.double()
    Hq, d = q.shape
    n, Hkv = k.shape[:2]
    zero = lambda x: x.unflatten(-1, (-1, 32)).amin(-1, keepdim=True).expand(n, Hkv, d // 32, 32).flatten(-2)  # noqa: E731
    zk, zv = zero(k), zero(v)
    out, bound = torch.zeros(2, Hq, d, dtype=torch.float64, device=q.device)
    rest = v - zv
    s_max = rest[seen].amax(0).unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1) / 15 / v_scale   # of each group
    tiny = int(seen.sum()) * 2.0 ** -37 * (15 * s_max.clamp(min=1) * (1 + s_max) * v_scale + zv[seen].abs().amax(0))
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        w = _weights(q[h], k[:, kv], scale, seen)[:, None]
        o = (w * v[:, kv]).sum(0)
        reach = float((((k - zk).abs() + zk.abs())[seen][:, kv] @ q[h].abs()).max()) * abs(scale)
        lam = 2 * P64.logit_slack(reach, d) + 2.0 ** -19
        dev, codes = (w * (v[:, kv] - o).abs()).sum(0), (w * rest[:, kv]).sum(0)
        mag = (w * (zv[:, kv].abs() + rest[:, kv])).sum(0)
        out[h] = o
        bound[h] = 1.01 * ((2.0 ** -11 + lam) * dev + 2.0 ** -11 * codes + (unit / 16 + 8) * 2.0 ** -22 * mag +
                           2.0 ** -8 * o.abs()) + tiny[kv]
    return out, bound


def decode(q, k, v, bs, scale, v_scale=1.0, window=0, sinks=0, part=0):
    """One sequence: written into a shuffled 4-bit pool, decoded; the output
    and the values the cache stands for."""
    n, Hkv, d = k.shape
    nb = -(-n // bs)
    kc, vc = (torch.full_like(pkv.make_kv4_cache(nb + 1, bs, Hkv, d), 0xFF) for _ in range(2))
    ids = torch.randperm(nb, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = ids[t // bs] * bs + t % bs
    pkv.paged_kv4_write(k, v, kc, vc, slots, bs, 1.0, v_scale)
    ks, vs = torch.empty(2, n, Hkv, d, device="cuda")
    pkv.paged_kv4_read(ks, vs, kc, vc, slots, bs, 1.0, v_scale)
    out = torch.empty_like(q)
    pkv.paged_attention_decode_kv4(out[None], q[None], kc, vc, ids.int()[None].contiguous(),
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), n, scale, bs, window, sinks,
                                   1.0, v_scale, part)
    return out, ks, vs


def _normal(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


@pytest.mark.parametrize("size", [1e-4, 1e-3, 1e-2, 1.0, 300.0, 1e4])
@pytest.mark.parametrize("spread", [2.0, 3.0])
@pytest.mark.parametrize("n,part,d,bs", [(8192, 0, 128, 16), (8192, -1, 128, 32), (8192, -1, 64, 16),
                                         (32768, -1, 128, 16)])
def test_values_of_every_size_under_peaked_weights(size, spread, n, part, d, bs):
    """Most tokens weigh a thousandth of the heaviest or less, together as much as it or more."""
    k, v, q = _normal(1, n, 2, d), size * _normal(2, n, 2, d), (spread * _normal(3, 8, d)).bfloat16()
    out, ks, vs = decode(q, k, v, bs, d ** -0.5, part=part)
    seen = torch.ones(n, dtype=torch.bool, device="cuda")
    ref, bound = reference(q, ks, vs, seen, d ** -0.5, 1.0, n if part else 1024)
    P64.assert_within(out, ref, bound)


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
@pytest.mark.parametrize("part", [0, -1, 128])
@pytest.mark.parametrize("d,bs", [(128, 16), (128, 32), (64, 16), (64, 32)])
def test_groups_and_tokens_of_different_sizes(window, sinks, part, d, bs):
    """Groups of 32 values from a thousandth to 10,000, a few tokens a hundred times the others (first, inside and
    last in a unit), a tensor scale other than 1."""
    n = 2001
    v = _normal(5, n, 2, d) * torch.tensor([1e-3, 1.0, 50.0, 1e4], device="cuda").repeat(d // 64)[:d // 32].repeat_interleave(32)
    v[[0, 3, 700, 1400, 1999, 2000]] *= 5.0
    v[1900:1940, 1] *= 100.0
    k, q = _normal(6, n, 2, d), (2 * _normal(7, 6, d)).bfloat16()
    out, ks, vs = decode(q, k, v, bs, d ** -0.5, 0.25, window, sinks, part)
    seen = P64.window_seen(n, n - 1, window, sinks)
    ref, bound = reference(q, ks, vs, seen, d ** -0.5, 0.25, n)
    P64.assert_within(out, ref, bound)


@pytest.mark.parametrize("n,part,drop", [(2049, 0, STAGE), (4096, 128, STAGE), (40000, 0, 1024)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_heavy_token_per_stage(n, part, drop, d):
    """Every stage (of the longest: every 1,024 tokens) holds one token with most of its weight: the bound holds, and
    refuses zeros and each output that leaves one such piece out."""
    u = _normal(1, 2, d)
    k, v = 0.1 * _normal(2, n, 2, d), _normal(3, n, 2, d)
    heavy = torch.arange(0, n, drop, device="cuda")
    heavy = (heavy + torch.randint(0, drop, heavy.shape, device="cuda",
                                   generator=torch.Generator(device="cuda").manual_seed(4))).clamp(max=n - 1)
    k[heavy] += u
    # the logit of a heavy token: 12 above the others'
    q = (12 * d ** 0.5 * u / (u * u).sum(-1, keepdim=True)).repeat_interleave(4, 0)
    q = (q + 0.05 * _normal(5, 8, d)).bfloat16()
    out, ks, vs = decode(q, k, v, 16, d ** -0.5, part=part)
    seen = torch.ones(n, dtype=torch.bool, device="cuda")
    ref, bound = reference(q, ks, vs, seen, d ** -0.5, 1.0, 1024)
    P64.assert_within(out, ref, bound)
    # the planted mistakes, in 64 bits on the host
    ref, bound, q, ks, vs, seen = (x.cpu() for x in (ref, bound, q, ks, vs, seen))
    assert ((ref.abs() > bound).double().mean(-1) > 0.7).all()
    for lo in range(0, n, max(drop, n // 16 // drop * drop)):
        less = seen.clone()
        less[lo:lo + drop] = False
        for h in range(0, 8, 3):
            w = _weights(q[h], ks[:, h // 4], d ** -0.5, less)
            wrong = (w[:, None] * vs[:, h // 4].double()).sum(0)
            assert ((wrong - ref[h]).abs() > bound[h]).double().mean() > 0.5, (lo, h)
