"""One workspace, made for the largest call of a loop, serves the smaller
ones, whose own choice of partitions may want more; nothing behind it is
written."""
import random

import pytest
import torch

from tests import plain64 as P64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

D, BS, HKV = 128, 16, 2
GUARD = 4096


class Guarded:
    """`n` zeroed bytes with bytes behind them that must stay as they are."""

    def __init__(self, n):
        self.all = torch.full((n + GUARD,), 0xAB, dtype=torch.uint8, device="cuda")
        self.ws = self.all[:n]
        self.ws.zero_()

    def check(self):
        assert (self.all[-GUARD:] == 0xAB).all()
        assert not self.ws[:16].any()                      # the counters are back at zero


def _pool(n, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-n // BS)
    k, v = (torch.randn(nb, BS, HKV, D, device="cuda", generator=g) for _ in range(2))
    return k, v, torch.randperm(nb, device="cuda", generator=g).int()


def _lens(rng, S, n):
    return [n] + [rng.randint(0, n) for _ in range(S - 1)]


def _check(out, q, k, v, ids, n, window, sinks, extra=0.0):
    """One row against 64 bits; weights of 8 bits, as the coarsest of the kernels rounds them (4 bits: `extra`)."""
    t = torch.arange(n, device="cuda")
    rows = (ids[t // BS].long() * BS + t % BS)
    kk, vv = k.flatten(0, 1)[rows], v.flatten(0, 1)[rows]
    o, _, mix, reach = P64.attend(q, kk, vv, P64.window_seen(n, n - 1, window, sinks), D ** -0.5)
    P64.assert_within(out, o, P64.out_bound(o, mix, 4 * reach, D, 2.0 ** -8, 2.0 ** -8, extra))


@pytest.mark.parametrize("kind,window,sinks", [("bf16", 4096, 0), ("e4m3", 4096, 0), ("f32", 4096, 0), ("kv4", 0, 0),
                                               ("scored", 0, 0), ("bf16", 1024, 4), ("kv4", 1024, 4)])
def test_decodes(kind, window, sinks):
    smax, nmax, Hq = 64, 4096, 12
    sizes = (lambda S, n: pkv.scored_workspace_size(S, Hq, HKV, D, BS, n)) if kind == "scored" else \
        (lambda S, n: pkv.decode_window_workspace_size(S, Hq, HKV, D, BS, n, window, sinks))
    room = Guarded(sizes(smax, nmax))
    k, v, ids = _pool(nmax)
    if kind == "kv4":
        kc, vc = (pkv.make_kv4_cache(ids.numel(), BS, HKV, D) for _ in range(2))
        every = torch.arange(nmax, device="cuda")
        pkv.paged_kv4_write(k.flatten(0, 1), v.flatten(0, 1), kc, vc, every, BS)
        k, v = torch.empty_like(k), torch.empty_like(v)
        pkv.paged_kv4_read(k.flatten(0, 1), v.flatten(0, 1), kc, vc, every, BS)
    else:
        kc, vc = (x.to({"e4m3": torch.float8_e4m3fn, "f32": torch.float32}.get(kind, torch.bfloat16)) for x in (k, v))
        k, v = kc.float(), vc.float()
    rng = random.Random(7)
    shapes = [(smax, nmax), (smax, 3000), (smax, 1000), (62, 4096), (1, 4096), (3, 500), (17, 2100), (40, 1500)]
    shapes += [(rng.randint(1, smax), rng.randint(1, nmax)) for _ in range(20)]
    more = 0
    for S, n in shapes:
        more += sizes(S, n) > room.ws.numel()
        lens = _lens(rng, S, n)
        tables = ids[None, :].expand(S, -1).contiguous()
        c = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = torch.randn(S, Hq, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)).bfloat16()
        out = torch.full_like(q, float("nan"))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(workspace=room.ws, err_word=err)
        if kind == "scored":
            t = torch.arange(nmax, device="cuda")
            slots = (tables[:, t // BS] * BS + t % BS).int().contiguous()
            scores = torch.zeros(S, nmax, device="cuda")
            pkv.token_attention_decode_scored(out, q, kc, vc, slots, c, scores, n, D ** -0.5, **kw)
            full = torch.tensor([Hq if m else 0 for m in lens], dtype=torch.float64, device="cuda")
            # a row's weights sum to 1, each off by its logit's error (below 2^-12 here) and a few roundings
            assert ((scores.double().sum(1) - full).abs() <= Hq * 2.0 ** -11).all()
        elif kind == "kv4":
            pkv.paged_attention_decode_kv4(out, q, kc, vc, tables, c, n, D ** -0.5, BS, window, sinks, **kw)
        else:
            pkv.paged_attention_decode_window(out, q, kc, vc, tables, c, n, D ** -0.5, window, sinks, **kw)
        assert int(err) == 0
        # 4-bit: the scale's product rounded too, of codes and zeros up to four times the largest value
        extra = 2.0 ** -9 * float(v.abs().max()) if kind == "kv4" else 0.0
        for s in {0, S - 1}:
            if lens[s]:
                _check(out[s], q[s], k, v, ids, lens[s], window, sinks, extra)
            else:
                assert (out[s] == 0).all()
        room.check()
    assert more or window == 1024                          # some smaller call's own choice wants more than there is


def test_query_chunks():
    window, sinks, Hq = 1024, 4, 14
    smax, qmax, nmax = 16, 512, 8192
    T = smax * qmax
    size = lambda S, t, ql, n: pkv.prefill_window_workspace_size(S, t, ql, Hq, HKV, D, BS, n, window, sinks)  # noqa: E731
    room = Guarded(size(smax, T, qmax, nmax))
    k, v, ids = _pool(nmax)
    kc, vc = k.bfloat16(), v.bfloat16()
    k, v = kc.float(), vc.float()
    rng, more = random.Random(5), 0
    shapes = [(16, 512, 8192), (1, 128, 8192), (1, 256, 8192), (2, 5, 3000), (1, 1, 4000), (4, 100, 1000), (16, 1, 8192)]
    shapes += [(rng.randint(1, 6), ql, rng.randint(ql, nmax)) for ql in [rng.randint(1, 300) for _ in range(12)]]
    for S, ql, n in shapes:
        t = S * ql
        more += size(S, t, ql, n) > room.ws.numel()
        lens = [n] + [rng.randint(ql, n) for _ in range(S - 1)]
        tables = ids[None, :].expand(S, -1).contiguous()
        q = torch.randn(t, Hq, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)).bfloat16()
        out, err = torch.full_like(q, float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")
        start = (torch.arange(S + 1, device="cuda") * ql).int()
        pkv.paged_attention_prefill_window(out, q, kc, vc, tables, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                           start, ql, n, D ** -0.5, window, sinks, workspace=room.ws, err_word=err)
        assert int(err) == 0
        for s in {0, S - 1}:
            for i in {0, ql // 2, ql - 1}:
                pos = lens[s] - ql + i
                _check(out[s * ql + i], q[s * ql + i], k, v, ids, pos + 1, window, sinks)
        room.check()
    assert more


def test_a_missing_workspace_or_one_short_of_a_request_is_refused():
    """The caller's own partition is not replaced, and a workspace without a header is none."""
    k, v, ids = _pool(1000)
    q = torch.randn(1, 12, D, device="cuda").bfloat16()
    args = (torch.empty_like(q), q, k.bfloat16(), v.bfloat16(), ids[None].contiguous(),
            torch.tensor([1000], dtype=torch.int32, device="cuda"), 1000, 0.1, 900, 4)
    for ws, part in ((torch.zeros(1024, dtype=torch.uint8, device="cuda"), 64), (torch.zeros(128, dtype=torch.uint8, device="cuda"), 0)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.paged_attention_decode_window(*args, partition_size=part, workspace=ws)
        assert e.value.status == 3
