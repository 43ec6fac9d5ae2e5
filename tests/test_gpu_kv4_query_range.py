"""Queries of any size in the 4-bit decode: the softmax depends on scale * q
alone, so a query times a power of two with the scale divided by it gives the
same bits."""
import pytest
import torch

from tests import plain64 as P64
from tests.test_gpu_kv4_accuracy import reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

N, HKV, BS = 700, 2, 16


def _cache(d):
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = torch.randn(2, N, HKV, d, device="cuda", generator=g)
    nb = -(-N // BS)
    kc, vc = (pkv.make_kv4_cache(nb, BS, HKV, d) for _ in range(2))
    slots = torch.arange(N, device="cuda")
    pkv.paged_kv4_write(k, v, kc, vc, slots, BS)
    ks, vs = torch.empty(2, N, HKV, d, device="cuda")
    pkv.paged_kv4_read(ks, vs, kc, vc, slots, BS)
    return kc, vc, torch.arange(nb, device="cuda").int()[None], ks, vs


def _decode(q, kc, vc, tables, scale, part):
    out = torch.full_like(q, 9.0)
    pkv.paged_attention_decode_kv4(out[None], q[None], kc, vc, tables, torch.tensor([N], dtype=torch.int32, device="cuda"),
                                   N, scale, BS, partition_size=part)
    return out


@pytest.mark.parametrize("d,Hq", [(128, 12), (64, 20)])
@pytest.mark.parametrize("part", [0, -1])
@pytest.mark.parametrize("power", [-60, -25, 11, 14, 40, 80])
def test_a_power_of_two_moves_between_query_and_scale(d, Hq, part, power):
    kc, vc, tables, ks, vs = _cache(d)
    q = torch.randn(Hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).bfloat16()
    base = _decode(q, kc, vc, tables, 0.125, part)
    ref, bound = reference(q, ks, vs, torch.ones(N, dtype=torch.bool, device="cuda"), 0.125, 1.0, N)
    P64.assert_within(base, ref, bound)
    for sign in (1.0, -1.0):
        got = _decode(q * (sign * 2.0 ** power), kc, vc, tables, sign * 0.125 * 2.0 ** -power, part)
        assert torch.equal(got, base)


@pytest.mark.parametrize("d", [64, 128])
def test_heads_of_different_sizes(d):
    """Of the eight heads of a unit, one 2^15 times the others' size, one zero, one not finite (NaN in it alone)."""
    kc, vc, tables, ks, vs = _cache(d)
    q = torch.randn(16, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    q[2] *= 2.0 ** 15
    q[5] = 0.0
    q[6, 7] = float("inf")
    q[9] *= 5000.0
    q = q.bfloat16()
    for scale in (0.125, 0.125 * 2.0 ** -15):
        out = _decode(q, kc, vc, tables, scale, 0)
        assert out[6].isnan().all()
        rest = [h for h in range(16) if h != 6]
        ref, bound = reference(q[rest[:7] + [0] + rest[7:]], ks, vs, torch.ones(N, dtype=torch.bool, device="cuda"), scale,
                               1.0, N)
        P64.assert_within(out[rest], torch.cat([ref[:7], ref[8:]]), torch.cat([bound[:7], bound[8:]]))
