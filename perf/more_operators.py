"""Cases that measure a prompt's way into the paged cache and the decode of
sequences that share one, with their plain forms: the rotary embedding with
the write of K and V into their slots, attention over whole packed prompts,
and the decode over block tables whose first blocks several sequences share.

`own` false: elementary torch operations in 32 bits.  `own` true: the calls of
paged_kv_cache_44_gb300.  `exact` gives the same results in 64 bits.
"""
import math
import random

import torch

own = False

LOWEST = float("-inf")
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 64 sequences: Q and K rotated, 64 new tokens into their slots; latency
        dict(name="rotary-step", kind="rotary", T=64, Hq=12, Hkv=2, d=128, rot=128, bs=16, f32=False, cache="bf16",
             packed=True, interleaved=False, far=4096, run=1, keep=False),
        # the tokens of 16 chunks and their decoding neighbours, rotated K kept for the chunk's own attention
        dict(name="rotary-prompt", kind="rotary", T=8240, Hq=28, Hkv=4, d=128, rot=128, bs=16, f32=False, cache="bf16",
             packed=True, interleaved=False, far=8192, run=512, keep=True),
        # a large prefill batch into an E4M3 cache, half of each head rotated, pairs side by side
        dict(name="rotary-e4m3", kind="rotary", T=16384, Hq=64, Hkv=8, d=128, rot=64, bs=32, f32=False, cache="e4m3",
             packed=False, interleaved=True, far=131072, run=4096, keep=False),
        # one short prompt: latency
        dict(name="prompt-one", kind="prompt", S=1, Hq=12, Hkv=2, d=128, lo=301, hi=301, klo=0, khi=0, causal=True,
             window=0, sinks=0),
        # 64 prompts of ragged lengths, packed
        dict(name="prompt-ragged", kind="prompt", S=64, Hq=28, Hkv=4, d=128, lo=1, hi=2048, klo=0, khi=0, causal=True,
             window=0, sinks=0),
        # one long document
        dict(name="prompt-long", kind="prompt", S=1, Hq=28, Hkv=4, d=128, lo=32768, hi=32768, klo=0, khi=0,
             causal=True, window=0, sinks=0),
        # both directions: encoder inputs of an embedding service, heads of 64, no sharing of K and V
        dict(name="prompt-encoder", kind="prompt", S=32, Hq=12, Hkv=12, d=64, lo=128, hi=1024, klo=0, khi=0,
             causal=False, window=0, sinks=0),
        # long prompts under a window with sinks
        dict(name="prompt-window", kind="prompt", S=8, Hq=64, Hkv=8, d=128, lo=4096, hi=8192, klo=0, khi=0,
             causal=True, window=1024, sinks=4),
        # the last few tokens of two long inputs: few rows, many keys
        dict(name="prompt-few-rows", kind="prompt", S=2, Hq=12, Hkv=2, d=128, lo=5, hi=9, klo=16384, khi=32768,
             causal=True, window=0, sinks=0),
        # eight samples of one short prompt
        dict(name="shared-small", kind="shared", G=1, M=8, P=304, lo=1, hi=40, alone=0, alo=0, ahi=0, Hq=12, Hkv=2,
             d=128, bs=16),
        # 100 of 256 requests with the same system prompt of 1,024 tokens
        dict(name="shared-prompt", kind="shared", G=1, M=100, P=1024, lo=1, hi=7168, alone=156, alo=1, ahi=8192, Hq=28,
             Hkv=4, d=128, bs=16),
        # four documents of 32,768 tokens, 16 questions about each
        dict(name="shared-documents", kind="shared", G=4, M=16, P=32768, lo=16, hi=1024, alone=0, alo=0, ahi=0, Hq=64,
             Hkv=8, d=128, bs=16),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["rotary", "rotary", "prompt", "prompt", "prompt", "shared", "shared"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    heads = dict(Hq=Hkv * rng.choice([1, 2, 4, 6, 7, 8, 10]), Hkv=Hkv, d=rng.choice([64, 128]))
    if kind == "rotary":
        T = _log(rng, 1, 16384)
        while T * heads["Hq"] > 1 << 20:
            T //= 2
        return dict(kind=kind, T=T, rot=rng.choice([heads["d"], heads["d"] // 2, 32]), bs=rng.choice([16, 32]),
                    f32=rng.random() < 0.3, cache=rng.choice(["f32", "bf16", "e4m3"]), packed=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, far=_log(rng, 1, 131072), run=rng.choice([1, 37, 512]),
                    keep=rng.random() < 0.5, **heads)
    if kind == "shared":
        G, M, P = _log(rng, 1, 4), _log(rng, 1, 64), _log(rng, 1, 32768)
        alone, hi, ahi = rng.choice([0, _log(rng, 1, 64)]), _log(rng, 1, 2048), _log(rng, 1, 8192)
        while (G * M * (P + hi) + alone * ahi) * heads["Hq"] > 1 << 27:
            M, P, alone = max(1, M // 2), max(1, P // 2), alone // 2
        return dict(kind=kind, G=G, M=M, P=P, lo=rng.randint(1, hi), hi=hi, alone=alone,
                    alo=rng.randint(1, ahi) if alone else 0, ahi=ahi if alone else 0, bs=rng.choice([16, 32]), **heads)
    S, hi = _log(rng, 1, 64), _log(rng, 1, 16384)
    khi = rng.choice([0, 0, _log(rng, hi, 32768)])
    while S * hi * max(hi, khi) * heads["Hq"] * heads["d"] > 1 << 40:
        S, hi = max(1, S // 2), max(1, hi // 2)
    causal = rng.random() < 0.75
    window = rng.choice([0, 0, _log(rng, 1, 16384)]) if causal else 0
    return dict(kind=kind, S=S, lo=_log(rng, 1, hi), hi=hi, klo=rng.randint(hi, khi) if khi >= hi else 0,
                khi=khi if khi >= hi else 0, causal=causal, window=window,
                sinks=rng.choice([0, 1, 4, 33, 128]) if window else 0, **heads)


def _ragged(n, lo, hi, what):
    """n lengths, uniform in [lo, hi], the first one hi: fixed by the case."""
    r = random.Random("%s %d %d %d" % (what, n, lo, hi))
    return ([hi] + [r.randint(lo, hi) for _ in range(n - 1)])[:n]


def _prompt_lengths(case):
    ql = _ragged(case["S"], case["lo"], case["hi"], "queries")
    return ql, (_ragged(case["S"], case["klo"], case["khi"], "keys") if case["khi"] else ql)


def _shared_lengths(case):
    """The shared length (whole blocks), the members' lengths and those of the sequences that share nothing."""
    P = case["P"] // case["bs"] * case["bs"]
    return (P, [P + t for t in _ragged(case["G"] * case["M"], case["lo"], case["hi"], "tails")],
            _ragged(case["alone"], case["alo"], case["ahi"], "alone"))


def _pairs(ql, kl, causal, window, sinks):
    """(query, key) pairs that are seen."""
    if not causal:
        return ql * kl
    seen = 0
    first = kl - ql
    if window <= 0:
        lo = max(first, 0)
        return (lo + 1 + kl) * (kl - lo) // 2 if kl > lo else 0
    for p in range(max(first, 0), kl):
        n = p + 1
        seen += n if n <= window else window + min(sinks, n - window)
    return seen


def work(case):
    kind, Hq, Hkv, d = case["kind"], case["Hq"], case["Hkv"], case["d"]
    if kind == "rotary":
        T, b = case["T"], 4 if case["f32"] else 2
        cb = {"f32": 4, "bf16": 2, "e4m3": 1}[case["cache"]]
        per = (Hq + 2 * Hkv) * d * b + case["rot"] * 4 + 16 + Hq * d * b + 2 * Hkv * d * cb
        return {"bytes": T * (per + (Hkv * d * b if case["keep"] else 0)), "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    if kind == "prompt":
        ql, kl = _prompt_lengths(case)
        pairs = sum(_pairs(q, k, case["causal"], case["window"], case["sinks"]) for q, k in zip(ql, kl))
        return {"bytes": 4 * sum(ql) * Hq * d + 4 * sum(kl) * Hkv * d, "flops": 4 * pairs * Hq * d}
    P, members, alone = _shared_lengths(case)
    tokens = case["G"] * P + sum(n - P for n in members) + sum(alone)
    S = len(members) + len(alone)
    return {"bytes": 4 * tokens * Hkv * d + 4 * S * Hq * d + 4 * (tokens // case["bs"] + S),
            "flops": 4 * (sum(members) + sum(alone)) * Hq * d}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _prepare_rotary(case, st, g):
    T, Hq, Hkv, d, bs, rot = (case[k] for k in ("T", "Hq", "Hkv", "d", "bs", "rot"))
    dt = torch.float32 if case["f32"] else torch.bfloat16
    if case["packed"]:
        # what one projection leaves: the heads of Q, K and V side by side in a token's row
        rows = _normal(g, T, Hq + 2 * Hkv, d).to(dt)
        st["q"], st["k"], st["v"] = rows.split([Hq, Hkv, Hkv], 1)
    else:
        st["q"], st["k"], st["v"] = (_normal(g, T, h, d).to(dt) for h in (Hq, Hkv, Hkv))
    # runs of consecutive tokens, each in shuffled blocks of its own and from a position of its own
    run, far = case["run"], case["far"]
    runs, per = -(-T // run), -(-run // bs)
    NB = runs * per + 1
    order = torch.randperm(NB - 1, device="cuda", generator=g) + 1
    i = torch.arange(T, device="cuda")
    st["slots"] = order[(i // run) * per + (i % run) // bs] * bs + (i % run) % bs
    start = torch.randint(0, far, (runs,), device="cuda", generator=g)
    st["positions"] = (start[i // run] + i % run) % far
    # the table a model makes once: cosines, then sines, of position * frequency, in 64 bits first
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * freq[None, :]
    st["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    cdt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3}[case["cache"]]
    st["kc"], st["vc"] = (torch.zeros(NB, bs, Hkv, d, device="cuda").to(cdt) for _ in range(2))
    st["k_scale"], st["v_scale"] = (6.0 / 448, 5.0 / 448) if cdt == E4M3 else (1.0, 1.0)
    st["q_out"] = torch.zeros(T, Hq, d, dtype=dt, device="cuda")
    st["k_out"] = torch.zeros(T, Hkv, d, dtype=dt, device="cuda") if case["keep"] else None


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _prepare_prompt(case, st, g):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    ql, kl = _prompt_lengths(case)
    st["ql"], st["kl"], st["scale"] = ql, kl, d ** -0.5
    st["q"] = _normal(g, sum(ql), Hq, d).bfloat16()
    st["k"], st["v"] = (_normal(g, sum(kl), Hkv, d).bfloat16() for _ in range(2))
    st["q_start"], st["k_start"] = _starts(ql), _starts(kl)
    st["out"] = torch.zeros_like(st["q"])
    if own:
        import paged_kv_cache_44_gb300 as pkv
        st["ws"] = pkv.make_prompt_workspace(case["S"], sum(ql), max(ql), max(kl), Hq, Hkv, d, case["window"],
                                             case["sinks"])


def _prepare_shared(case, st, g):
    Hq, Hkv, d, bs, G, M = (case[k] for k in ("Hq", "Hkv", "d", "bs", "G", "M"))
    P, members, alone = _shared_lengths(case)
    lens, head = members + alone, P // bs
    S, MB = len(lens), max(-(-n // bs) for n in lens)
    own_blocks = [-(-n // bs) - (head if s < G * M else 0) for s, n in enumerate(lens)]
    NB = G * head + sum(own_blocks) + 1
    order = (torch.randperm(NB - 1, device="cuda", generator=g) + 1).to(torch.int32)
    tables = torch.zeros(S, MB, dtype=torch.int32, device="cuda")
    at = 0
    for s in range(G * M):
        tables[s, :head] = order[s // M * head:(s // M + 1) * head]
    at = G * head
    for s, n in enumerate(own_blocks):
        lo = head if s < G * M else 0
        tables[s, lo:lo + n] = order[at:at + n]
        at += n
    st["tables"], st["n"], st["lens"] = tables, torch.tensor(lens, dtype=torch.int32, device="cuda"), lens
    # the groups follow one another; the sequences that share nothing are the last group
    starts = [i * M for i in range(G + 1)] + ([S] if alone else [])
    shared = [P] * G + ([0] if alone else [])
    st["group_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["shared"] = torch.tensor(shared, dtype=torch.int32, device="cuda")
    st["bounds"] = (max(lens), P, M)
    st["scale"] = d ** -0.5
    st["q"] = _normal(g, S, Hq, d).bfloat16()
    st["kc"], st["vc"] = (_normal(g, NB, bs, Hkv, d).bfloat16() for _ in range(2))
    st["out"] = torch.zeros_like(st["q"])
    if own:
        import paged_kv_cache_44_gb300 as pkv
        st["ws"] = pkv.make_shared_workspace(S, len(shared), Hq, Hkv, d, bs, *st["bounds"])


def prepare(case, seed):
    g, st = _gen(seed), dict(case)
    {"rotary": _prepare_rotary, "prompt": _prepare_prompt, "shared": _prepare_shared}[case["kind"]](case, st, g)
    return st


# -------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, d] with its first rot values rotated by cos, sin [T, rot / 2], in 32 bits."""
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    a, b = (head[..., ::2], head[..., 1::2]) if interleaved else head.chunk(2, -1)
    cos, sin = cos[:, None], sin[:, None]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((head, rest), -1)


def _stored(x, dtype, by):
    if dtype != E4M3:
        return x.to(dtype)
    return (x / torch.full((), by, device=x.device)).clamp(-448, 448).to(E4M3)


def _plain_rotary(st):
    cos, sin = st["cos_sin"][st["positions"]].chunk(2, -1)
    q, k = (_rotate(st[x], cos, sin, st["rot"], st["interleaved"]) for x in ("q", "k"))
    Hkv, d, dt = st["Hkv"], st["d"], st["q"].dtype
    for x, c, by in ((k, "kc", "k_scale"), (st["v"].float(), "vc", "v_scale")):
        rows = _stored(x, st[c].dtype, st[by])
        raw = torch.uint8 if rows.dtype == E4M3 else rows.dtype
        st[c].view(raw).view(-1, Hkv, d)[st["slots"]] = rows.view(raw)
    return [q.to(dt)] + ([k.to(dt)] if st["keep"] else []) + [st["kc"], st["vc"]]


def _soft(q, k, v, hidden, scale):
    """q [r, d], k and v [n, d], hidden [r, n] or None: softmax(q k) v, zeros where nothing is seen, in the inputs' type."""
    x = (q @ k.T) * scale
    if hidden is not None:
        x = x.masked_fill(hidden, LOWEST)
    w = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    return (w @ v) / w.sum(-1, keepdim=True).clamp(min=1e-300 if q.dtype == torch.float64 else 1e-38)


def _prompt(st, dtype, out):
    """Whole prompts, head by head and some rows at a time."""
    g, q0, k0 = st["Hq"] // st["Hkv"], 0, 0
    for ql, kl in zip(st["ql"], st["kl"]):
        step = max(1, (1 << 27) // kl)
        t = torch.arange(kl, device="cuda")
        for r in range(0, ql, step):
            m = min(step, ql - r)
            hidden = None
            if st["causal"]:
                p = kl - ql + torch.arange(r, r + m, device="cuda")[:, None]
                hidden = t[None, :] > p
                if st["window"] > 0:
                    hidden |= (t[None, :] <= p - st["window"]) & (t[None, :] >= st["sinks"])
            for h in range(st["Hq"]):
                k, v = (st[x][k0:k0 + kl, h // g].to(dtype) for x in ("k", "v"))
                out[q0 + r:q0 + r + m, h] = _soft(st["q"][q0 + r:q0 + r + m, h].to(dtype), k, v, hidden,
                                                  st["scale"]).to(out.dtype)
        q0, k0 = q0 + ql, k0 + kl
    return out


def _plain_shared(st):
    """Every sequence on its own, as a decode without sharing does it."""
    bs, Hkv, d = st["bs"], st["Hkv"], st["d"]
    out = torch.empty_like(st["q"])
    for s, n in enumerate(st["lens"]):
        ids = st["tables"][s, :-(-n // bs)].long()
        k, v = (st[c][ids].flatten(0, 1)[:n].float().transpose(0, 1) for c in ("kc", "vc"))
        x = (st["q"][s].float().view(Hkv, -1, d) @ k.transpose(1, 2)) * st["scale"]
        w = torch.exp(x - x.amax(-1, keepdim=True))
        out[s] = ((w @ v) / w.sum(-1, keepdim=True)).view(-1, d).to(out.dtype)
    return [out]


def run(state):
    st, kind = state, state["kind"]
    if not own:
        if kind == "rotary":
            return _plain_rotary(st)
        return [_prompt(st, torch.float32, torch.empty_like(st["q"]))] if kind == "prompt" else _plain_shared(st)
    import paged_kv_cache_44_gb300 as pkv
    if kind == "rotary":
        pkv.rotary_kv_write(st["q"], st["k"], st["v"], st["positions"], st["cos_sin"], st["q_out"], st["k_out"],
                            st["kc"], st["vc"], st["slots"], interleaved=st["interleaved"], k_scale=st["k_scale"],
                            v_scale=st["v_scale"])
        return [st["q_out"]] + ([st["k_out"]] if st["keep"] else []) + [st["kc"], st["vc"]]
    if kind == "prompt":
        pkv.prompt_attention(st["out"], st["q"], st["k"], st["v"], st["q_start"], max(st["ql"]), st["scale"],
                             key_start=st["k_start"], max_key_len=max(st["kl"]), causal=st["causal"],
                             window=st["window"], num_sinks=st["sinks"], workspace=st["ws"])
        return [st["out"]]
    pkv.paged_attention_decode_shared(st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["n"],
                                      st["group_start"], st["shared"], *st["bounds"], scale=st["scale"],
                                      workspace=st["ws"])
    return [st["out"]]


# -------------------------------------------------------------------- exact

def _exact_rotary(st):
    T, rot, Hkv, d = st["T"], st["rot"], st["Hkv"], st["d"]
    pos = st["cos_sin"].double()[st["positions"]]
    half = rot // 2
    j = torch.arange(half, device="cuda")
    lo, hi = (2 * j, 2 * j + 1) if st["interleaved"] else (j, j + half)
    turned = []
    for x in ("q", "k"):
        y = st[x].double().clone()
        z = torch.complex(y[:, :, lo], y[:, :, hi]) * torch.complex(pos[:, :half], pos[:, half:])[:, None]
        y[:, :, lo], y[:, :, hi] = z.real, z.imag
        turned.append(y)
    q, k = turned
    pools = []
    for x, c, by in ((k, "kc", "k_scale"), (st["v"].double(), "vc", "v_scale")):
        pool = torch.zeros(st[c].shape, dtype=torch.float64, device="cuda")
        if st[c].dtype == E4M3:
            x = (x / float(torch.tensor(st[by], dtype=torch.float32))).clamp(-448, 448)
        blocks, offs = st["slots"] // st["bs"], st["slots"] % st["bs"]
        pool[blocks, offs] = x
        pools.append(pool)
    return [q] + ([k] if st["keep"] else []) + pools


def exact(case, seed):
    st, kind = prepare(case, seed), case["kind"]
    if kind == "rotary":
        return _exact_rotary(st)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    g = Hq // Hkv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    if kind == "shared":
        for s, n in enumerate(st["lens"]):
            t = torch.arange(n, device="cuda")
            slot = st["tables"][s, t // case["bs"]].long() * case["bs"] + t % case["bs"]
            for kv in range(Hkv):
                k, v = (st[c].view(-1, Hkv, d)[slot, kv].double() for c in ("kc", "vc"))
                p = torch.softmax(st["q"][s, kv * g:kv * g + g].double() @ k.T * st["scale"], -1)
                out[s, kv * g:kv * g + g] = p @ v
        return [out]
    if 4 * Hq * d * sum(a * b for a, b in zip(st["ql"], st["kl"])) > 6e12:
        return None
    qs, ks = st["q_start"].tolist(), st["k_start"].tolist()
    for s in range(case["S"]):
        ql, kl = qs[s + 1] - qs[s], ks[s + 1] - ks[s]
        for r in range(0, ql, 2048):
            rows = torch.arange(r, min(ql, r + 2048), device="cuda")
            far = (kl - ql + rows)[:, None] - torch.arange(kl, device="cuda")[None, :]   # how far back a key lies
            seen = torch.ones_like(far, dtype=torch.bool)
            if case["causal"]:
                seen = far >= 0
                if case["window"] > 0:
                    seen &= (far < case["window"]) | (torch.arange(kl, device="cuda") < case["sinks"])[None, :]
            empty = ~seen.any(-1)
            for h in range(Hq):
                k, v = (st[x][ks[s]:ks[s + 1], h // g].double() for x in ("k", "v"))
                logit = st["q"][qs[s] + rows, h].double() @ k.T * st["scale"]
                p = torch.softmax(logit.masked_fill(~seen, LOWEST), -1)
                p[empty] = 0
                out[qs[s] + rows, h] = p @ v
    return [out]
