"""Cases that measure the 4-bit cache, the windowed attention and the
eviction operators of paged_kv_cache_44_gb300, with their plain forms.

`own` false: elementary torch operations in 32 bits.  `own` true: the
library's calls.  `exact` gives the same results in 64 bits.
"""
import random

import torch

own = False

GROUP = 32            # values of a 4-bit row that share a scale and a zero
HALF_MAX = 65504.0
LOWEST = float("-inf")


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 64 sequences: 64 new tokens quantised into their slots and read back
        dict(name="kv4-write-step", kind="kv4_rw", T=64, Hkv=2, d=128, bs=16, f32=False, run=1),
        # a prompt chunk of 8,192 tokens, stored block by block
        dict(name="kv4-write-prompt", kind="kv4_rw", T=8192, Hkv=8, d=128, bs=16, f32=False, run=512),
        # one short sequence on the 4-bit cache: latency
        dict(name="kv4-decode-one", kind="kv4", S=1, Hq=12, Hkv=2, d=128, bs=16, lo=301, hi=301, window=0, sinks=0),
        # the long-context decode, every sequence 32,768 tokens, 4-bit cache
        dict(name="kv4-decode-long", kind="kv4", S=32, Hq=64, Hkv=8, d=128, bs=16, lo=32768, hi=32768, window=0,
             sinks=0),
        # fp32 cache, a few tokens of window: the smallest windowed call
        dict(name="window-decode-f32", kind="window", cache="f32", S=4, Hq=4, Hkv=2, d=64, bs=16, lo=2, hi=53,
             window=16, sinks=4),
        # 256 sequences of ragged lengths that keep a window of 1,024 and four sinks
        dict(name="window-decode-bf16", kind="window", cache="bf16", S=256, Hq=28, Hkv=4, d=128, bs=16, lo=1, hi=8192,
             window=1024, sinks=4),
        # E4M3 cache, blocks of 32, a wide window
        dict(name="window-decode-e4m3", kind="window", cache="e4m3", S=128, Hq=28, Hkv=4, d=128, bs=32, lo=256,
             hi=16384, window=4096, sinks=64),
        # 512-token chunks of 16 prompts under the same window
        dict(name="window-prefill", kind="prefill", S=16, ql=512, Hq=28, Hkv=4, d=128, bs=16, lo=512, hi=8192,
             window=1024, sinks=4),
        # a decoding step that also accumulates the attention weights
        dict(name="scored-decode-bf16", kind="scored", cache="bf16", S=64, Hq=12, Hkv=2, d=128, bs=16, lo=512, hi=4096),
        # the same on an E4M3 cache and longer sequences
        dict(name="scored-decode-e4m3", kind="scored", cache="e4m3", S=32, Hq=28, Hkv=4, d=128, bs=16, lo=256,
             hi=16384),
        # a few short sequences cut to 512 tokens
        dict(name="evict-small", kind="evict", S=4, lo=300, hi=1000, budget=512, first=4, recent=128),
        # 64 long sequences cut to 4,096 tokens
        dict(name="evict-long", kind="evict", S=64, lo=16384, hi=32768, budget=4096, first=4, recent=1024),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["kv4_rw", "kv4", "kv4", "window", "window", "prefill", "scored", "evict"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    heads = dict(Hq=Hkv * rng.choice([1, 2, 4, 6, 7, 8, 10]), Hkv=Hkv, d=rng.choice([64, 128]),
                 bs=rng.choice([16, 32]))
    if kind == "kv4_rw":
        heads.pop("Hq")
        return dict(kind=kind, T=_log(rng, 1, 8192), f32=rng.random() < 0.5, run=rng.choice([1, 37, 512]), **heads)
    if kind == "evict":
        hi = _log(rng, 8, 32768)
        budget = _log(rng, 1, hi)
        first = min(rng.choice([0, 1, 4, 17]), budget)
        return dict(kind=kind, S=_log(rng, 1, 64), lo=_log(rng, 1, hi), hi=hi, budget=budget, first=first,
                    recent=rng.randint(0, budget - first))
    if kind == "prefill":
        ql = _log(rng, 1, 512)
        hi = _log(rng, ql, 8192)
        S = _log(rng, 1, 8)
        while S * ql * heads["Hq"] * hi > 1 << 27:
            S, ql = max(1, S // 2), max(1, ql // 2)
        return dict(kind=kind, S=S, ql=ql, lo=rng.randint(ql, hi), hi=hi, window=_log(rng, 1, 8192),
                    sinks=rng.choice([0, 1, 4, 33, 128]), **heads)
    S = _log(rng, 1, 64)
    hi = _log(rng, 1, 32768)
    while S * hi * Hkv > 1 << 20:
        hi //= 2
    lens = dict(S=S, lo=_log(rng, 1, hi), hi=hi)
    if kind == "kv4":
        window = rng.choice([0, _log(rng, 1, 32768)])
        return dict(kind=kind, window=window, sinks=rng.choice([0, 1, 4, 33]) if window else 0, **lens, **heads)
    if kind == "window":
        return dict(kind=kind, cache=rng.choice(["f32", "bf16", "e4m3"]), window=_log(rng, 1, 32768),
                    sinks=rng.choice([0, 1, 4, 33, 128]), **lens, **heads)
    return dict(kind=kind, cache=rng.choice(["bf16", "e4m3"]), **lens, **heads)


def _lengths(case):
    """Sequence lengths, uniform in [lo, hi], the first one hi: fixed by the case."""
    r = random.Random("%d %d %d" % (case["S"], case["lo"], case["hi"]))
    return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["S"] - 1)]


def _visible(n, window, sinks):
    return n if window <= 0 or n <= window else window + min(sinks, n - window)


def work(case):
    kind = case["kind"]
    if kind == "kv4_rw":
        rows, d = 2 * case["T"] * case["Hkv"], case["d"]
        row4 = d // 2 + d // 8
        # written: values in, rows out; read back: rows in, fp32 values out
        return {"bytes": rows * ((4 if case["f32"] else 2) * d + 2 * row4 + 4 * d) + 16 * case["T"],
                "flops": 8 * rows * d}
    ns = _lengths(case)
    if kind == "evict":
        kept = [min(n, case["budget"]) for n in ns]
        return {"bytes": sum(8 * n + 8 * k + 4 * (n - k) for n, k in zip(ns, kept)) + 8 * len(ns), "flops": sum(ns)}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if kind == "prefill":
        ql, w, sinks = case["ql"], case["window"], case["sinks"]
        pairs = sum(_visible(n - ql + i + 1, w, sinks) for n in ns for i in range(ql))
        # keys that some query of the chunk sees: the sinks and the span of the windows
        keys = sum(min(n, w + ql - 1 + sinks) for n in ns)
        return {"bytes": 4 * len(ns) * ql * Hq * d + keys * Hkv * d * 4, "flops": 4 * pairs * Hq * d}
    row = {"kv4": d // 2 + d // 8, "f32": 4 * d, "bf16": 2 * d, "e4m3": d}[case.get("cache", "kv4")]
    tokens = sum(_visible(n, case.get("window", 0), case.get("sinks", 0)) for n in ns)
    qbytes = (8 if case.get("cache") == "f32" else 4) * len(ns) * Hq * d
    extra = 12 * tokens if kind == "scored" else 0       # slot, score in, score out
    return {"bytes": 2 * row * Hkv * tokens + qbytes + extra, "flops": 4 * tokens * Hq * d}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _tables(ns, bs, g):
    """Block tables [S, MB] over a shuffled pool whose block 0 is in no table, the lengths and the pool's size."""
    blocks = torch.tensor([-(-n // bs) for n in ns], device="cuda")
    total, MB = int(blocks.sum()), max(1, int(blocks.max()))
    order = (torch.randperm(total, device="cuda", generator=g) + 1).to(torch.int32)
    used = torch.arange(MB, device="cuda")[None, :] < blocks[:, None]
    tables = torch.zeros(len(ns), MB, dtype=torch.int32, device="cuda")
    tables[used] = order
    return tables, torch.tensor(ns, dtype=torch.int32, device="cuda"), total + 1


def _kv4_random(NB, bs, Hkv, d, g):
    """K and V pools of the 4-bit format with random codes and the scales and zeros that N(0, 1) values have."""
    rows = bs * d // 2
    pools = []
    for _ in range(2):
        pool = torch.randint(0, 256, (NB, Hkv, bs * (d // 2 + d // 8)), dtype=torch.uint8, device="cuda", generator=g)
        n = bs * d // GROUP
        scale = 0.2 + 0.15 * torch.rand(NB, Hkv, n, device="cuda", generator=g)
        zero = -8.0 * scale + 0.3 * _normal(g, NB, Hkv, n)
        pool[..., rows:rows + 2 * n] = scale.half().view(torch.uint8)
        pool[..., rows + 2 * n:] = zero.half().view(torch.uint8)
        pools.append(pool)
    return pools


def _pools(cache, NB, bs, Hkv, d, g):
    """K and V pools of one of the other formats and their scales."""
    k, v = _normal(g, NB, bs, Hkv, d), _normal(g, NB, bs, Hkv, d)
    if cache == "f32":
        return k, v, 1.0, 1.0
    if cache == "bf16":
        return k.bfloat16(), v.bfloat16(), 1.0, 1.0
    ks, vs = 5.5 / 448, 5.0 / 448
    return ((k / ks).clamp(-448, 448).to(torch.float8_e4m3fn), (v / vs).clamp(-448, 448).to(torch.float8_e4m3fn), ks,
            vs)


def prepare(case, seed):
    g, kind = _gen(seed), case["kind"]
    st = dict(case)
    if kind == "kv4_rw":
        T, Hkv, d, bs = case["T"], case["Hkv"], case["d"], case["bs"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        st["key"], st["value"] = _normal(g, T, Hkv, d).to(dt), _normal(g, T, Hkv, d).to(dt)
        # runs of consecutive tokens, each in shuffled blocks of its own
        run = case["run"]
        per = -(-run // bs)
        NB = -(-T // run) * per + 1
        order = torch.randperm(NB - 1, device="cuda", generator=g) + 1
        i = torch.arange(T, device="cuda")
        st["slots"] = order[(i // run) * per + (i % run) // bs] * bs + (i % run) % bs
        size = (NB, Hkv, bs * (d // 2 + d // 8))
        st["kc"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        st["vc"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        st["k_out"], st["v_out"] = torch.zeros(2, T, Hkv, d, device="cuda")
        st["k_scale"], st["v_scale"] = 1.0, 0.75
        return st
    ns = _lengths(case)
    if kind == "evict":
        S, MT = len(ns), max(ns)
        st["n"] = torch.tensor(ns, dtype=torch.int32, device="cuda")
        st["slots"] = torch.randperm(S * MT, device="cuda", generator=g).view(S, MT).to(torch.int32)
        # accumulated weights: most tokens light, a few heavy, and ties among those never attended
        u = torch.rand(S, MT, device="cuda", generator=g)
        st["scores"] = torch.where(u < 0.05, torch.zeros_like(u), u ** 4 * 20)
        st["new_slots"] = torch.full((S, MT), -1, dtype=torch.int32, device="cuda")
        st["new_scores"] = torch.zeros(S, MT, device="cuda")
        st["new_n"] = torch.zeros(S, dtype=torch.int32, device="cuda")
        st["evicted"] = torch.full((S, MT), -1, dtype=torch.int32, device="cuda")
        return st
    Hq, Hkv, d, bs, S = case["Hq"], case["Hkv"], case["d"], case["bs"], case["S"]
    st["scale"], st["max"] = d ** -0.5, max(ns)
    st["tables"], st["n"], NB = _tables(ns, bs, g)
    qdt = torch.float32 if case.get("cache") == "f32" else torch.bfloat16
    rows = S * case["ql"] if kind == "prefill" else S
    st["q"] = _normal(g, rows, Hq, d).to(qdt)
    st["out"] = torch.zeros(rows, Hq, d, dtype=qdt, device="cuda")
    if kind == "kv4":
        st["kc"], st["vc"] = _kv4_random(NB, bs, Hkv, d, g)
        st["k_scale"], st["v_scale"] = 1.0, 0.75
    else:
        st["kc"], st["vc"], st["k_scale"], st["v_scale"] = _pools(case.get("cache", "bf16"), NB, bs, Hkv, d, g)
    if kind == "prefill":
        st["start"] = (torch.arange(S + 1, device="cuda") * case["ql"]).to(torch.int32)
    if kind == "scored":
        t = torch.arange(st["max"], device="cuda")
        st["slots"] = (st["tables"][:, t // bs] * bs + (t % bs)[None, :]).to(torch.int32)
        st["scores"] = torch.rand(S, st["max"], device="cuda", generator=g)
    if own:
        # the workspace a serving loop allocates once and passes to every call
        import paged_kv_cache_44_gb300 as pkv
        shape = (S, Hq, Hkv, d, bs, st["max"])
        if kind == "prefill":
            st["ws"] = pkv.make_prefill_window_workspace(S, rows, case["ql"], Hq, Hkv, d, bs, st["max"],
                                                         case["window"], case["sinks"])
        elif kind == "scored":
            st["ws"] = pkv.make_scored_workspace(*shape)
        else:
            st["ws"] = pkv.make_window_workspace(*shape, case["window"], case["sinks"])
    return st


# -------------------------------------------------------------- plain forms

def _kv4_unpack(pool, bs, d, transposed):
    """fp32 values [..., bs, d] of 4-bit block rows [..., bs * (d/2 + d/8)]: K rows, or V rows (transposed)."""
    lead, G, n = pool.shape[:-1], d // GROUP, bs * d // GROUP
    code, par = pool[..., :bs * d // 2], pool[..., bs * d // 2:].contiguous().view(torch.float16).float()
    code = torch.stack((code & 15, code >> 4), -1)
    if not transposed:
        code = code.reshape(*lead, bs, 4, G, 8).transpose(-3, -2).reshape(*lead, bs, G, GROUP)
        scale, zero = par[..., :n].reshape(*lead, bs, G, 1), par[..., n:].reshape(*lead, bs, G, 1)
    else:
        # [tile, half, r, c, group, parity, nibble] -> token (tile, half, c, parity), value (group, r, nibble)
        k = len(lead)
        code = code.reshape(*lead, bs // 16, 2, 8, 4, G, 2, 4)
        code = code.permute(*range(k), k, k + 1, k + 3, k + 5, k + 4, k + 2, k + 6).reshape(*lead, bs, G, GROUP)
        par = par.reshape(*lead, 2, bs // 2, G, 2).transpose(-2, -1).reshape(*lead, 2, bs, G, 1)
        scale, zero = par[..., 0, :, :, :], par[..., 1, :, :, :]
    return (code.float() * scale + zero).reshape(*lead, bs, d)


def _kv4_rows(x, by):
    """The values that 4-bit rows of x [..., d] stand for."""
    y = (x.float() / torch.full((), by, device=x.device)).clamp(-HALF_MAX, HALF_MAX)
    y = y.unflatten(-1, (-1, GROUP))
    zero = y.amin(-1, keepdim=True).half().float()
    top = (y.amax(-1, keepdim=True) - zero).clamp(min=0)
    step = (top / torch.full((), 15.0, device=x.device)).half().float()
    code = torch.where(step > 0, torch.round((y - zero) / step).clamp(0, 15), torch.zeros_like(y))
    return ((zero + step * code) * by).flatten(-2)


def _gathered(st):
    """K and V [S, n, Hkv, d] in fp32, read through the block tables."""
    t, bs, d = st["tables"].long(), st["bs"], st["d"]
    if st["kind"] == "kv4":
        k, v = (_kv4_unpack(st[c][t], bs, d, c == "vc").transpose(2, 3) for c in ("kc", "vc"))
    else:
        k, v = st["kc"][t].float(), st["vc"][t].float()
    return k.flatten(1, 2) * st["k_scale"], v.flatten(1, 2) * st["v_scale"]


def _attend(q, k, v, seen, scale):
    """q [S, Q, Hq, d], k/v [S, n, Hkv, d], seen [S, Q, n]: outputs [S, Q, Hq, d] and weights [S, Hkv, g, Q, n]."""
    S, Q, Hq, d = q.shape
    n, Hkv = k.shape[1], k.shape[2]
    qg = q.float().reshape(S, Q, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, d)
    x = (qg @ k.permute(0, 2, 3, 1)) * scale
    x = x.view(S, Hkv, Hq // Hkv, Q, n).masked_fill(~seen[:, None, None], LOWEST)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    o = w.reshape(S, Hkv, -1, n) @ v.permute(0, 2, 1, 3)
    return o.view(S, Hkv, Hq // Hkv, Q, d).permute(0, 3, 1, 2, 4).reshape(S, Q, Hq, d), w


def _seen(st, n_keys, Q):
    """[S, Q, n]: key t is seen by query i at position p when t <= p and (t < sinks or t > p - window)."""
    t = torch.arange(n_keys, device="cuda")[None, None, :]
    p = (st["n"][:, None].long() - Q + torch.arange(Q, device="cuda")[None, :])[:, :, None]
    ok = t <= p
    if st.get("window", 0) > 0:
        ok &= (t < st["sinks"]) | (t > p - st["window"])
    return ok


def _plain(st):
    kind = st["kind"]
    if kind == "kv4_rw":
        return [_kv4_rows(st["key"], st["k_scale"]), _kv4_rows(st["value"], st["v_scale"])]
    if kind == "evict":
        slots, scores, n = st["slots"], st["scores"], st["n"].long()[:, None]
        S, MT = slots.shape
        t = torch.arange(MT, device="cuda")[None, :].expand(S, MT)
        kept_n = n.clamp(max=st["budget"])
        rank = torch.where((t < st["first"]) | (t >= n - st["recent"]), float("inf"), scores)
        rank = torch.where(t < n, rank, LOWEST)
        order = torch.argsort(rank, dim=1, descending=True, stable=True)
        place = torch.empty_like(order).scatter_(1, order, t)
        keep = (place < kept_n) & (t < n)
        gone = ~keep & (t < n)
        new_slots, new_scores, out = st["new_slots"].clone(), st["new_scores"].clone(), st["evicted"].clone()
        to, away = (keep.cumsum(1) - 1)[keep], (gone.cumsum(1) - 1)[gone]
        row = torch.arange(S, device="cuda")[:, None].expand(S, MT)
        new_slots[row[keep], to] = slots[keep]
        new_scores[row[keep], to] = scores[keep]
        out[row[gone], away] = slots[gone]
        return [new_slots, new_scores, kept_n[:, 0].int(), out]
    k, v = _gathered(st)
    Q = st.get("ql", 1)
    q = st["q"].view(st["S"], Q, st["Hq"], st["d"])
    seen = _seen(st, k.shape[1], Q)
    o, w = _attend(q, k, v, seen, st["scale"])
    o = o.reshape(st["q"].shape).to(st["q"].dtype)
    if kind != "scored":
        return [o]
    st["scores"] += w.sum((1, 2, 3))[:, :st["max"]]
    return [o, st["scores"]]


def run(state):
    if not own:
        return _plain(state)
    import paged_kv_cache_44_gb300 as pkv
    st, kind = state, state["kind"]
    if kind == "kv4_rw":
        pkv.paged_kv4_write(st["key"], st["value"], st["kc"], st["vc"], st["slots"], st["bs"], k_scale=st["k_scale"],
                            v_scale=st["v_scale"])
        pkv.paged_kv4_read(st["k_out"], st["v_out"], st["kc"], st["vc"], st["slots"], st["bs"], k_scale=st["k_scale"],
                           v_scale=st["v_scale"])
        return [st["k_out"], st["v_out"]]
    if kind == "evict":
        pkv.evict_tokens(st["slots"], st["scores"], st["n"], st["new_slots"], st["new_scores"], st["new_n"],
                         budget=st["budget"], num_first=st["first"], num_recent=st["recent"], evicted=st["evicted"])
        return [st["new_slots"], st["new_scores"], st["new_n"], st["evicted"]]
    more = dict(scale=st["scale"], workspace=st["ws"])
    if kind == "kv4":
        pkv.paged_attention_decode_kv4(st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["n"], st["max"],
                                       block_size=st["bs"], window=st["window"], num_sinks=st["sinks"],
                                       k_scale=st["k_scale"], v_scale=st["v_scale"], **more)
    elif kind == "window":
        pkv.paged_attention_decode_window(st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["n"], st["max"],
                                          window=st["window"], num_sinks=st["sinks"], k_scale=st["k_scale"],
                                          v_scale=st["v_scale"], **more)
    elif kind == "prefill":
        pkv.paged_attention_prefill_window(st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["n"], st["start"],
                                           st["ql"], st["max"], window=st["window"], num_sinks=st["sinks"], **more)
    else:
        pkv.token_attention_decode_scored(st["out"], st["q"], st["kc"], st["vc"], st["slots"], st["n"], st["scores"],
                                          st["max"], k_scale=st["k_scale"], v_scale=st["v_scale"], **more)
        return [st["out"], st["scores"]]
    return [st["out"]]


# -------------------------------------------------------------------- exact

def _single(x):
    """64-bit values rounded to the nearest fp32, for a format whose definition names fp32 operations."""
    return x.to(torch.float32).double()


def _exact_rows(x, by):
    by = float(torch.tensor(by, dtype=torch.float32))
    y = _single(x.double() / by).clamp(-HALF_MAX, HALF_MAX)
    out = torch.empty_like(y)
    for lo in range(0, y.shape[-1], GROUP):
        part = y[..., lo:lo + GROUP]
        zero = part.min(-1).values.to(torch.float32).half().double()
        reach = _single((part.max(-1).values - zero).clamp(min=0))
        step = _single(reach / 15).to(torch.float32).half().double()
        safe = torch.where(step > 0, step, torch.ones_like(step))
        code = torch.round(_single(_single(part - zero[..., None]) / safe[..., None])).clamp(0, 15)
        code = torch.where((step > 0)[..., None], code, torch.zeros_like(code))
        out[..., lo:lo + GROUP] = _single(zero[..., None] + step[..., None] * code) * by
    return out


def _exact_block_values(pool, blocks, bs, d, value):
    """[blocks * bs, Hkv, d] values of 4-bit blocks, each found by its place: byte and nibble of its code, scale, zero."""
    raw = pool[blocks.long()]
    t = torch.arange(bs, device="cuda")[:, None]
    e = torch.arange(d, device="cuda")[None, :]
    G, grp = d // GROUP, e // GROUP
    if not value:
        nib = 8 * (t * 4 * G + (e % GROUP) // 8 * G + grp) + e % 8
        par = t * G + grp
    else:
        tile, k = t // 16, t % 16
        word = ((tile * 2 + k // 8) * 8 + (e % GROUP) // 4) * 4 * G + (k // 2 % 4) * G + grp
        nib = 8 * word + 4 * (k % 2) + e % 4
        par = ((tile * 8 + k // 2) * G + grp) * 2 + k % 2
    code = (raw[..., nib // 2].int() >> (4 * (nib % 2))) & 15
    halves = raw[..., bs * d // 2:].contiguous().view(torch.float16).double()
    val = halves[..., par] * code + halves[..., par + bs * G]
    return val.permute(0, 2, 1, 3).reshape(-1, pool.shape[1], d)


def exact(case, seed):
    st, kind = prepare(case, seed), case["kind"]
    if kind == "kv4_rw":
        return [_exact_rows(st["key"], st["k_scale"]), _exact_rows(st["value"], st["v_scale"])]
    if kind == "evict":
        moved = st["new_scores"].double().cpu()
        for s, n in enumerate(st["n"].tolist()):
            sc = st["scores"][s, :n].double().cpu().tolist()
            keep = range(n)
            if n > case["budget"]:
                fixed = set(range(case["first"])) | set(range(n - case["recent"], n))
                rest = sorted((i for i in range(n) if i not in fixed), key=lambda i: (-sc[i], i))
                keep = sorted(fixed | set(rest[:case["budget"] - len(fixed)]))
            moved[s, :len(keep)] = torch.tensor([sc[i] for i in keep], dtype=torch.float64)
        return [None, moved.cuda(), None, None]
    S, Hq, Hkv, d, bs = case["S"], case["Hq"], case["Hkv"], case["d"], case["bs"]
    Q = case.get("ql", 1)
    out = torch.zeros(S, Q, Hq, d, dtype=torch.float64, device="cuda")
    added = st["scores"].double() if kind == "scored" else None
    ks, vs = (float(torch.tensor(st[c], dtype=torch.float32)) for c in ("k_scale", "v_scale"))
    for s, n in enumerate(st["n"].tolist()):
        blocks = st["tables"][s, :-(-n // bs)]
        if kind == "kv4":
            k, v = (_exact_block_values(st[c], blocks, bs, d, c == "vc")[:n] for c in ("kc", "vc"))
        else:
            k, v = (st[c][blocks.long()].double().reshape(-1, Hkv, d)[:n] for c in ("kc", "vc"))
        pos = torch.arange(n - Q, n, device="cuda")
        far = pos[:, None] - torch.arange(n, device="cuda")[None, :]
        hidden = far < 0
        if case.get("window", 0) > 0:
            hidden |= (far >= case["window"]) & (torch.arange(n, device="cuda")[None, :] >= case["sinks"])
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            logit = st["q"].view(S, Q, Hq, d)[s, :, h].double() @ (k[:, kv].T * ks) * st["scale"]
            p = torch.softmax(logit.masked_fill(hidden, LOWEST), -1)
            out[s, :, h] = p @ (v[:, kv] * vs)
            if added is not None:
                added[s, :n] += p[0]
    out = out.view(st["q"].shape)
    return [out, added] if kind == "scored" else [out]
