"""Arguments the windowed, 4-bit and eviction calls refuse, on the host: no
GPU is needed, and a call that got past its checks would answer 4 here."""
import ctypes
import inspect
import struct

import pytest
import torch

import paged_kv_cache_44_gb300 as pkv

A = 1 << 20            # an aligned address nothing reads
OK_SHAPE = dict(S=2, MB=64, max=1000, Hq=8, Hkv=2, d=128, bs=16, NB=100)


def _window(kernel=0, window=64, sinks=4, part=0, q=1, c=1, out=A, query=A, ws=0, wsb=0, scale=0.1, ks=1.0, vs=1.0, **kw):
    s = {**OK_SHAPE, **kw}
    return pkv.lib.pkv_paged_attention_decode_window(out, query, q, A, A, c, A, s["MB"], A, s["S"], s["max"], s["Hq"],
                                                     s["Hkv"], s["d"], s["bs"], s["NB"], scale, ks, vs, window, sinks,
                                                     part, ws or None, wsb, None, None, kernel)


def _kv4(window=64, sinks=4, part=0, q=1, out=A, ws=0, wsb=0, scale=0.1, ks=1.0, vs=1.0, **kw):
    s = {**OK_SHAPE, **kw}
    return pkv.lib.pkv_paged_attention_decode_kv4(out, A, q, A, A, A, s["MB"], A, s["S"], s["max"], s["Hq"], s["Hkv"],
                                                  s["d"], s["bs"], s["NB"], scale, ks, vs, window, sinks, part,
                                                  ws or None, wsb, None, None)


COMMON = [(dict(Hq=7), 1), (dict(d=96), 2), (dict(bs=8), 2), (dict(S=-1), 1), (dict(S=65536), 2), (dict(max=1025), 1),
          (dict(NB=0), 1), (dict(out=A + 8), 1), (dict(out=None), 1), (dict(part=-2), 1), (dict(part=24), 1),
          (dict(scale=float("nan")), 1), (dict(sinks=-1), 1), (dict(part=16), 3), (dict(part=16, ws=A, wsb=300), 3),
          (dict(part=16, ws=A + 8, wsb=1 << 30), 1)]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(window=0), 1), (dict(window=-5), 1), (dict(q=2), 2), (dict(c=7), 2),
                                                (dict(kernel=3), 1), (dict(kernel=2, c=0), 2),
                                                (dict(c=2, ks=0.0), 1), (dict(c=2, vs=float("inf")), 1), (dict(S=0), 0)])
def test_window_decode(kw, status):
    assert _window(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [(dict(window=-1), 1), (dict(q=0), 2), (dict(ks=-1.0), 1),
                                                (dict(vs=float("nan")), 1), (dict(S=0), 0)])
def test_kv4_decode(kw, status):
    assert _kv4(**kw) == status


@pytest.mark.parametrize("kw,status", [(dict(window=0), 1), (dict(sinks=-1), 1), (dict(q=0), 2), (dict(c=2), 2),
                                       (dict(ql=2000), 1), (dict(part=16), 3), (dict(T=0), 0), (dict(d=32), 2),
                                       (dict(qs=A + 2), 1)])
def test_window_prefill(kw, status):
    s = {**OK_SHAPE, **dict(window=64, sinks=4, q=1, c=1, ql=100, T=150, part=0, qs=A), **kw}
    got = pkv.lib.pkv_paged_attention_prefill_window(A, A, s["q"], A, A, s["c"], A, s["MB"], A, s["qs"], s["S"], s["T"],
                                                     s["ql"], s["max"], s["Hq"], s["Hkv"], s["d"], s["bs"], s["NB"], 0.1,
                                                     s["window"], s["sinks"], s["part"], None, 0, None, None)
    assert got == status


@pytest.mark.parametrize("call", ["pkv_paged_kv4_write", "pkv_paged_kv4_read"])
@pytest.mark.parametrize("kw,status", [(dict(T=-1), 1), (dict(T=0), 0), (dict(dt=2), 2), (dict(d=96), 2), (dict(bs=8), 2),
                                       (dict(Hkv=0), 1), (dict(ks=0.0), 1), (dict(vs=float("inf")), 1), (dict(k=None), 1),
                                       (dict(k=A + 4), 1), (dict(slots=A + 4), 1), (dict(NB=0), 1)])
def test_kv4_rows(call, kw, status):
    s = {**dict(T=5, dt=1, NB=10, bs=16, Hkv=2, d=128, ks=1.0, vs=1.0, k=A, slots=A), **kw}
    assert getattr(pkv.lib, call)(s["k"], A, s["dt"], A, A, s["slots"], s["T"], s["NB"], s["bs"], s["Hkv"], s["d"],
                                  s["ks"], s["vs"], None, None) == status


@pytest.mark.parametrize("kw,status", [(dict(scores=None), 1), (dict(scores=A + 2), 1), (dict(max=1001), 1), (dict(c=0), 2),
                                       (dict(ws=None), 3), (dict(wsb=1000), 3), (dict(ws=A + 8), 1), (dict(S=0), 0),
                                       (dict(part=7), 1), (dict(max=-1), 1)])
def test_scored_decode(kw, status):
    s = {**OK_SHAPE, **dict(MT=1000, c=1, scores=A, ws=A, wsb=1 << 40, part=0), **kw}
    assert pkv.lib.pkv_token_attention_decode_scored(
        A, A, 1, A, A, s["c"], A, s["MT"], A, s["scores"], s["S"], s["max"], s["Hq"], s["Hkv"], s["d"], s["bs"], s["NB"],
        0.1, 1.0, 1.0, s["part"], s["ws"], s["wsb"], None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(S=0), 0), (dict(S=65536), 2), (dict(MT=0), 1), (dict(MT=(1 << 30) + 1), 2), (dict(budget=-1), 1), (dict(first=-1), 1),
    (dict(recent=-1), 1), (dict(first=50, recent=51), 1), (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1, budget=2 ** 31 - 1), 1),
    (dict(slots=None), 1), (dict(new_num=None), 1), (dict(new_slots=A), 1), (dict(new_slots=A + 2396), 1),
    (dict(new_scores=4 * A), 1), (dict(evicted=5 * A), 1), (dict(evicted=2 * A + 1200), 1), (dict(new_num=3 * A), 1),
    (dict(scores=2 * A + 1), 1), (dict(evicted=7 * A + 2), 1)])
def test_evict(kw, status):
    s = {**dict(slots=A, scores=2 * A, num=3 * A, S=2, MT=300, budget=100, first=4, recent=20, new_slots=4 * A,
                new_scores=5 * A, new_num=6 * A, evicted=7 * A), **kw}
    assert pkv.lib.pkv_evict_tokens(s["slots"], s["scores"], s["num"], s["S"], s["MT"], s["budget"], s["first"],
                                    s["recent"], s["new_slots"], s["new_scores"], s["new_num"], s["evicted"], None,
                                    None) == status


def test_workspace_sizes():
    f = pkv.decode_window_workspace_size
    whole = pkv.decode_workspace_size(32, 64, 8, 128, 16, 32768)
    assert f(32, 64, 8, 128, 16, 32768, 0) == whole                     # no window
    assert f(32, 64, 8, 128, 16, 32768, 2 ** 31 - 1, 2 ** 31 - 1) == whole
    assert 0 < f(32, 64, 8, 128, 16, 32768, 1024, 4) < whole
    assert f(32, 64, 8, 128, 16, 32768, -1) == 0 and f(32, 64, 8, 96, 16, 32768, 5) == 0
    g = pkv.prefill_window_workspace_size
    assert g(4, 100, 50, 8, 2, 128, 16, 1000, 0) == 0 and g(4, 100, 50, 8, 2, 128, 16, 1000, 64, -1) == 0
    assert g(4, 100, 50, 8, 0, 128, 16, 1000, 64) == 0
    assert g(4, 100, 50, 8, 2, 128, 16, 1000, 64, 4) >= 256
    h = pkv.scored_workspace_size
    # the decode's, and a float per token and head (heads of a set in pairs)
    base = pkv.decode_workspace_size(2, 14, 2, 128, 16, 1000)
    assert h(2, 14, 2, 128, 16, 1000) >= base + 4 * 2 * 2 * 8 * 1000
    assert h(2, 14, 3, 128, 16, 1000) == 0
    assert pkv.kv4_block_bytes(16, 2, 128) == 16 * 2 * 80 and pkv.kv4_block_bytes(32, 3, 64) == 32 * 3 * 40
    assert pkv.kv4_block_bytes(8, 2, 128) == 0 and pkv.kv4_block_bytes(16, 0, 128) == 0
    with pytest.raises(ValueError):
        pkv.make_kv4_cache(4, 16, 2, 96, device="cpu")


def test_binding_refuses_wrong_tensors():
    t = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    f32 = torch.float32
    with pytest.raises(ValueError):
        pkv.evict_tokens(t(2, 5), t(2, 5, dt=f32), t(2), t(2, 5), t(2, 6, dt=f32), t(2), 3)
    with pytest.raises(ValueError):
        pkv.evict_tokens(t(2, 5), t(2, 5), t(2), t(2, 5), t(2, 5, dt=f32), t(2), 3)
    kc = pkv.make_kv4_cache(4, 16, 2, 128, device="cpu")
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    for bad in (dict(value=x[:2]), dict(value=x.float()), dict(key_cache=kc[..., :-16]), dict(block_size=32),
                dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), dict(key_cache=kc[:, :1])):
        args = {**dict(key=x, value=x, key_cache=kc, value_cache=kc, slot_mapping=torch.zeros(3, dtype=torch.int64),
                       block_size=16), **bad}
        with pytest.raises(ValueError):
            pkv.paged_kv4_write(**args)
    # a layer cannot be decoded with tables of another batch
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.paged_attention_decode_kv4(torch.empty_like(q), q, kc, kc, t(1, 4), t(2), 10, 0.1, 16)


def test_binding_refuses_another_device(monkeypatch):
    """Tensors of a device that is not the current one, strided ones (no GPU is needed for either)."""
    class Elsewhere:
        device = torch.device("cuda", 1)
        get_device = staticmethod(lambda: 1)
        is_contiguous = staticmethod(lambda: False)
    for dev in (0, 1):
        monkeypatch.setattr(pkv, "_current_device", lambda: dev)
        assert pkv._pointers(3, None, None) == [0, 0, 3]
        with pytest.raises(ValueError, match="contiguous" if dev else "device"):
            pkv._pointers(None, Elsewhere(), None)
        with pytest.raises(ValueError, match="int32"):
            pkv._pointers(None, None, torch.zeros(4, dtype=torch.uint8))
    for call in (pkv.paged_attention_decode_window, pkv.paged_attention_prefill_window, pkv.paged_kv4_write,
                 pkv.paged_kv4_read, pkv.paged_attention_decode_kv4, pkv.token_attention_decode_scored,
                 pkv.evict_tokens):
        text = inspect.getsource(call)
        assert "_pointers(" in text and "_ptr(" not in text


def test_arguments_in_one_array():
    """pkv_invoke gives each call its arguments: refusals are the call's own, wherever the bad argument stands."""
    symbols = ["pkv_paged_attention_decode_window", "pkv_paged_attention_prefill_window", "pkv_paged_kv4_write",
               "pkv_paged_kv4_read", "pkv_paged_attention_decode_kv4", "pkv_token_attention_decode_scored",
               "pkv_evict_tokens"]
    good = [  # no sequences or tokens: accepted without a launch
        (0, 0, 1, 0, 0, 1, 0, 4, 0, 0, 64, 8, 2, 128, 16, 9, 0.1, 1.0, 1.0, 5, 4, 0, 0, 0, 0, 0, 0),
        (0, 0, 1, 0, 0, 1, 0, 4, 0, 0, 0, 0, 0, 64, 8, 2, 128, 16, 9, 0.1, 5, 4, 0, 0, 0, 0, 0),
        (0, 0, 1, 0, 0, 0, 0, 9, 16, 2, 128, 1.0, 1.0, 0, 0), (0, 0, 1, 0, 0, 0, 0, 9, 16, 2, 128, 1.0, 1.0, 0, 0),
        (0, 0, 1, 0, 0, 0, 4, 0, 0, 64, 8, 2, 128, 16, 9, 0.1, 1.0, 1.0, 5, 4, 0, 0, 0, 0, 0),
        (0, 0, 1, 0, 0, 1, 0, 64, 0, 0, 0, 64, 8, 2, 128, 16, 9, 0.1, 1.0, 1.0, 0, 0, 0, 0, 0),
        (0, 0, 0, 0, 7, 4, 1, 1, 0, 0, 0, 0, 0, 0)]
    for number, (symbol, args) in enumerate(zip(symbols, good)):
        f = getattr(pkv.lib, symbol)
        assert len(f.argtypes) == len(args)
        kinds = {ctypes.c_void_p: "Q", ctypes.c_int: "q", ctypes.c_float: "d", ctypes.c_size_t: "Q"}
        pack = struct.Struct("=" + "".join(kinds[t] for t in f.argtypes)).pack
        assert f(*args) == 0 and pkv.lib.pkv_invoke(number, pack(*args)) == 0
        refused = 0
        for i, t in enumerate(f.argtypes):
            for bad in {ctypes.c_int: (-7, 12345), ctypes.c_float: (float("nan"),)}.get(t, ()):
                other = args[:i] + (bad,) + args[i + 1:]
                want = f(*other)
                assert pkv.lib.pkv_invoke(number, pack(*other)) == want, (symbol, i, bad)
                refused += want != 0
            if t == ctypes.c_int:
                assert pkv.lib.pkv_invoke(number, pack(*args[:i], 1 << 32, *args[i + 1:])) == 1, (symbol, i)
        assert refused > 4
    assert pkv.lib.pkv_invoke(7, bytes(400)) == 1 and pkv.lib.pkv_invoke(-1, bytes(400)) == 1
    assert pkv.lib.pkv_invoke(0, None) == 1
