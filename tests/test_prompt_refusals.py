"""Arguments that the rotary write, the prompt attention and the shared decode
refuse, on the host: no GPU is needed, and a call that got past its checks
would answer 4 here."""
import pytest
import torch

import paged_kv_cache_44_gb300 as pkv

A = 1 << 30            # an aligned address nothing reads


def _rotary(q=A, k=2 * A, v=3 * A, dt=1, qs=1024, ks=256, vs=256, pos=4 * A, cs=5 * A, mp=100, rot=128, inter=0, qo=6 * A,
            qos=1024, ko=7 * A, kos=256, kc=8 * A, vc=9 * A, cdt=1, slots=10 * A, T=5, NB=10, bs=16, Hq=8, Hkv=2, d=128,
            k_scale=1.0, v_scale=1.0):
    return pkv.lib.pkv_rotary_kv_write(q, k, v, dt, qs, ks, vs, pos, cs, mp, rot, inter, qo, qos, ko, kos, kc, vc, cdt,
                                       slots, T, NB, bs, Hq, Hkv, d, k_scale, v_scale, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(T=0), 0), (dict(dt=2), 2), (dict(cdt=5), 2), (dict(d=120, rot=96), 2), (dict(d=528, qs=1 << 14, qos=1 << 14, ks=1 << 12, vs=1 << 12, kos=1 << 12), 2),
    (dict(rot=8), 2), (dict(rot=144), 1), (dict(rot=-16), 1), (dict(mp=0), 1), (dict(Hq=-1), 1), (dict(Hq=0), 1),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(slots=None), 1), (dict(pos=None), 1), (dict(cs=None), 1), (dict(q=A + 8), 1), (dict(qs=1023), 1), (dict(qs=1028), 1),
    (dict(ks=255), 1), (dict(kos=128), 1), (dict(cs=5 * A + 4), 1), (dict(pos=4 * A + 4), 1), (dict(NB=0), 1),
    (dict(cdt=2, k_scale=0.0), 1), (dict(cdt=2, v_scale=float("nan")), 1), (dict(kc=8 * A + 2), 1),
    # outputs over something else that is read or written
    (dict(qo=2 * A), 1), (dict(qo=A + 16), 1), (dict(qo=A, qos=2048), 1), (dict(ko=3 * A), 1), (dict(ko=6 * A + 256), 1),
    (dict(T=1 << 20, qs=1 << 30), 1), (dict(NB=1 << 30, bs=1 << 10), 1), (dict(qo=8 * A + 4096), 1), (dict(kc=9 * A), 1), (dict(qs=1536, q=A, k=A + 2048, ks=1536, qo=A + 1024, qos=1536), 1)])
def test_rotary(kw, status):
    assert _rotary(**kw) == status


def test_rotary_without_anything_to_do():
    none = dict(kc=None, vc=None, slots=None, v=None)
    assert _rotary(q=None, qo=None, Hq=0, k=None, ko=None, Hkv=0, **none) == 1
    assert _rotary(k=None, ko=None, Hkv=0, T=0, **none) == 0


def test_rotary_binding():
    x = torch.zeros(4, 2, 64)
    pos, cs = torch.zeros(4, dtype=torch.int64), torch.zeros(10, 64)
    for args, kw in [((x, None, None, pos, cs), {}), ((None, None, None, pos, cs), {}), ((x, x, None, pos, cs, x), {}),
                     ((x, None, None, pos.int(), cs, x), {}), ((x, None, None, pos, cs.double(), x), {}),
                     ((x, None, None, pos, cs, x.double()), {}), ((x, None, None, pos, cs, x[:3]), {}),
                     ((x, x, x, pos, cs, x, x), {}), ((x.transpose(1, 2), None, None, pos, cs, x.transpose(1, 2)), {})]:
        with pytest.raises((ValueError, TypeError)):
            pkv.rotary_kv_write(*args, **kw)


def _prompt(out=A, q=2 * A, k=3 * A, v=4 * A, dt=1, qs=1024, ks=256, vs=256, q_start=5 * A, k_start=6 * A, S=2, Tq=100,
            Tk=100, mq=60, mk=60, Hq=8, Hkv=2, d=128, scale=0.1, causal=1, window=0, sinks=0, part=0, ws=7 * A, wsb=1 << 40):
    return pkv.lib.pkv_prompt_attention(out, q, k, v, dt, qs, ks, vs, q_start, k_start, S, Tq, Tk, mq, mk, Hq, Hkv, d, scale,
                                        causal, window, sinks, part, ws, wsb, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(S=0), 0), (dict(S=65536), 2), (dict(Tq=0), 0), (dict(Tq=-1), 1), (dict(Tk=-1), 1), (dict(mq=-1), 1),
    (dict(mk=-1), 1), (dict(dt=0), 2), (dict(dt=2), 2), (dict(d=96), 2), (dict(Hq=7), 1), (dict(Hkv=0), 1),
    (dict(scale=float("inf")), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(window=5, causal=0), 1), (dict(part=-2), 1),
    (dict(part=100), 1), (dict(out=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(q_start=None), 1),
    (dict(k_start=None), 1), (dict(q=2 * A + 8), 1), (dict(qs=1020), 1), (dict(qs=1028), 1), (dict(ks=255), 1),
    (dict(vs=1 << 38), 1), (dict(out=A + 4), 1), (dict(q_start=5 * A + 2), 1), (dict(out=2 * A), 1), (dict(out=3 * A - 16), 1),
    (dict(out=4 * A + 2048), 1), (dict(Tq=(1 << 30) + 1), 2), (dict(Tk=(1 << 30) + 1), 2),
    (dict(vs=1 << 37, Tk=1 << 10), 1), (dict(part=128, mk=1000, ws=None, wsb=0), 3), (dict(part=128, mk=1000, wsb=1000), 3),
    (dict(part=128, mk=1000, ws=7 * A + 8), 1)])
def test_prompt(kw, status):
    assert _prompt(**kw) == status


def test_prompt_workspace():
    f = pkv.prompt_workspace_size
    assert f(2, 100, 60, 60, 8, 2, 128) == 256                           # a few stages are not split
    units = 9 * 12 * 8                                                   # 9 queries, 12 heads, 1,000 keys in 128s
    assert 256 + units * 130 * 4 <= f(2, 9, 5, 1000, 12, 2, 128, partition_size=128) < 256 + units * 130 * 4 + 1024
    assert f(2, 9, 5, 32768, 12, 2, 128) > 256                           # few rows over many keys
    assert f(2, 9, 5, 32768, 12, 2, 128, window=100, num_sinks=2) == 256
    assert f(2, 9, 5, 32768, 12, 2, 96) == 0 and f(2, 9, 5, 32768, 12, 5, 128) == 0 and f(2, 9, 5, 100, 12, 2, 128, -1) == 0
    assert f(2, 9, 5, 1000, 12, 2, 128, partition_size=64) == 0


def test_prompt_binding():
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    qs = torch.tensor([0, 4], dtype=torch.int32)
    for args, kw in [((q, q, k, k.float(), qs, 4, 1.0), {}), ((q, q, k, k[:3], qs, 4, 1.0), {}), ((q[:2], q, k, k, qs, 4, 1.0), {}),
                     ((q, q, k, k, qs.long(), 4, 1.0), {}), ((q, q, k, k, qs, 4, 1.0), dict(key_start=qs[:1], max_key_len=4)), ((q, q, k, k, qs, 4, 1.0), dict(key_start=qs)),
                     ((q, q, k, k, qs, 4, 1.0), dict(max_key_len=4))]:
        with pytest.raises(ValueError):
            pkv.prompt_attention(*args, workspace=q, **kw)


def _shared(out=A, q=2 * A, qd=1, kc=3 * A, vc=4 * A, cd=1, tables=5 * A, MB=100, lens=6 * A, gs=7 * A, sl=8 * A, S=4, G=2,
            mx=1000, ms=500, mg=3, Hq=8, Hkv=2, d=128, bs=16, NB=200, scale=0.1, part=0, ws=9 * A, wsb=1 << 40, sharing=1):
    return pkv.lib.pkv_paged_attention_decode_shared(out, q, qd, kc, vc, cd, tables, MB, lens, gs, sl, S, G, mx, ms, mg, Hq,
                                                     Hkv, d, bs, NB, scale, part, ws, wsb, None, None, sharing)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(S=0), 0), (dict(S=65536), 2), (dict(G=-1), 1), (dict(G=65536), 2), (dict(mx=1601), 1), (dict(ms=-1), 1),
    (dict(ms=1001), 1), (dict(mg=-1), 1), (dict(mg=65536), 2), (dict(qd=0), 2), (dict(cd=0), 2), (dict(cd=2), 2), (dict(d=96), 2),
    (dict(bs=8), 2), (dict(Hq=9), 1), (dict(NB=0), 1), (dict(scale=float("nan")), 1), (dict(part=-2), 1), (dict(part=24), 1),
    (dict(out=None), 1), (dict(lens=None), 1), (dict(gs=None), 1), (dict(sl=None), 1), (dict(gs=7 * A + 2), 1),
    (dict(sl=8 * A + 1), 1), (dict(kc=3 * A + 8), 1), (dict(sharing=2), 1), (dict(sharing=-1), 1), (dict(ws=None, wsb=0), 3),
    (dict(part=64, wsb=1000), 3), (dict(ws=9 * A + 8), 1)])
def test_shared(kw, status):
    assert _shared(**kw) == status


def test_shared_workspace():
    f = pkv.shared_workspace_size
    plain = pkv.decode_workspace_size(64, 64, 8, 128, 16, 33792)
    assert f(64, 4, 64, 8, 128, 16, 33792, 0, 0) == plain                     # nothing to share
    assert f(4, 1, 8, 2, 128, 16, 5000, 304, 4) == pkv.decode_workspace_size(4, 8, 2, 128, 16, 5000)
    assert f(4, 1, 8, 2, 128, 16, 500, 304, 4) == pkv.decode_window_workspace_size(4, 8, 2, 128, 16, 500, 500)
    assert f(4, 1, 8, 2, 128, 16, 500, 304, 4, sharing="always") >= 256 + 4 * 8 * 2 * 130 * 4
    assert f(64, 4, 64, 8, 128, 16, 33792, 32768, 16) > 64 * 64 * 2 * 130 * 4
    assert f(64, 4, 64, 8, 128, 16, 1000, 1001, 16) == 0 and f(64, -1, 64, 8, 128, 16, 1000, 100, 16) == 0
    assert f(64, 4, 64, 8, 96, 16, 1000, 100, 16) == 0 and f(64, 4, 64, 8, 128, 16, 1000, 100, 16, 10) == 0


def test_shared_binding():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kc, i = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    n, gs = i[0, :2].contiguous(), i[0, :3].contiguous()
    for args, kw in [((q, q, kc, kc[:4], i, n, gs, n, 10, 0, 0, 1.0), {}), ((q, q, kc, kc, i, n, gs, gs, 10, 0, 0, 1.0), {}),
                     ((q, q, kc, kc, i, n, gs.long(), n, 10, 0, 0, 1.0), {}), ((q, q, kc, kc, i[:1], n, gs, n, 10, 0, 0, 1.0), {}),
                     ((q.float(), q, kc, kc, i, n, gs, n, 10, 0, 0, 1.0), {}), ((q, q, kc, kc, i, n, gs, n, 10, 0, 0, 1.0), dict(sharing="no"))]:
        with pytest.raises(ValueError):
            pkv.paged_attention_decode_shared(*args, workspace=q, **kw)
