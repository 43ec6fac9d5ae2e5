"""An fp32 query over an E4M3 cache: the windowed decode, with its merge
inside the launch and after it, and the scored decode."""
import pytest
import torch

from tests import plain64 as P64
from tests.test_gpu_window import LENS, _pool

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

E4M3 = torch.float8_e4m3fn


def _bound(o, mix, reach, d, m, v):
    """The query is rounded to fp16 for the products, which moves a logit by 2^-11 of its magnitudes on either side of
    the division; the weights to fp16, those below its smallest normal number by 2^-25; the output to fp32."""
    small = m * 2.0 ** -25 * float(v.abs().max()) if m else 0.0
    return P64.out_bound(o, mix, reach, d, 2.0 ** -11 + 2 * 2.0 ** -11 * reach[:, None], 2.0 ** -24, small)


@pytest.mark.parametrize("shape", [(12, 2, 128, 16), (10, 1, 64, 32), (7, 7, 128, 32)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("window,sinks,part,copies", [(300, 5, 0, 1), (5000, 0, -1, 1), (200, 3, 64, 1), (200, 3, 64, 20),
                                                      (1500, 33, 128, 20)])
@pytest.mark.parametrize("kernel", ["auto", "cuda_cores"])
def test_window(shape, window, sinks, part, copies, kernel):
    """copies: few sets of heads, or more than the GPU has SMs (merged by a launch of their own)."""
    Hq, Hkv, d, bs = shape
    seen_of = lambda s, n: P64.window_seen(n, n - 1, window, sinks)  # noqa: E731
    (kc, vc), tables, dense, sc = _pool(LENS, Hkv, d, bs, E4M3, 3, seen_of)
    q = torch.randn(len(LENS), Hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    n = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    qs, ts, ns = q.repeat(copies, 1, 1), tables.repeat(copies, 1), n.repeat(copies)
    out, err = torch.full_like(qs, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode_window(out, qs, kc, vc, ts, ns, max(LENS), d ** -0.5, window, sinks, k_scale=sc, v_scale=sc,
                                      partition_size=part, err_word=err, kernel=kernel)
    assert int(err) == 0
    out = out.view(copies, len(LENS), Hq, d)
    for i in range(1, copies):
        assert torch.equal(out[i], out[0])
    for s, m in enumerate(LENS):
        o, _, mix, reach = P64.attend(q[s], dense[0][s], dense[1][s], seen_of(s, m), d ** -0.5)
        P64.assert_within(out[0, s], o, _bound(o, mix, reach, d, m, dense[1][s]), f"sequence {s} of {m}")


@pytest.mark.parametrize("Hq,Hkv,d,bs", [(12, 2, 128, 16), (7, 1, 64, 32), (3, 3, 128, 16), (10, 1, 64, 16)])
@pytest.mark.parametrize("part", [0, -1, 128])
def test_scored(Hq, Hkv, d, bs, part):
    lens = [0, 1, 33, 500, 2000]
    S, MT = len(lens), max(lens) + 5
    NB, sc = -(-S * MT // bs), 5.0 / 448
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = ((torch.randn(NB, bs, Hkv, d, device="cuda", generator=g) / sc).clamp(-448, 448).to(E4M3) for _ in range(2))
    slots = torch.randperm(NB * bs, device="cuda", generator=g)[:S * MT].view(S, MT).int()
    q = torch.randn(S, Hq, d, device="cuda", generator=g)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = torch.rand(S, MT, device="cuda", generator=g)
    scores, out, plain = before.clone(), torch.empty_like(q), torch.empty_like(q)
    kw = dict(scale=d ** -0.5, k_scale=sc, v_scale=sc, partition_size=part)
    pkv.token_attention_decode_scored(out, q, k, v, slots, n, scores, max(lens), **kw)
    if part != 0:
        pkv.token_attention_decode(plain, q, k, v, slots, n, max(lens), **kw)
        assert torch.equal(out, plain)
    for s, m in enumerate(lens):
        assert torch.equal(scores[s, m:], before[s, m:])
        idx = slots[s, :m].long()
        kk, vv = k.flatten(0, 1)[idx].double() * sc, v.flatten(0, 1)[idx].double() * sc
        o, w, mix, reach = P64.attend(q[s], kk, vv, torch.ones(m, dtype=torch.bool, device="cuda"), d ** -0.5)
        P64.assert_within(out[s], o, _bound(o, mix, reach, d, m, vv), f"output of {m}")
        rel = (2 * P64.logit_slack(reach, d) + 2 * 2.0 ** -11 * reach)[:, None] + 2.0 ** -19 + Hq * 2.0 ** -24
        want = before[s, :m].double() + w.sum(0)
        P64.assert_within(scores[s, :m], want, 1.01 * (rel * w).sum(0) + 2.0 ** -24 * want + 1e-30, f"scores of {m}")
