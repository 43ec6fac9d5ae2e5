"""Plain 64-bit forms for the tests of the windowed attention, the 4-bit
cache and the eviction calls: textbook definitions, written per sequence and
head, with the sums that the tolerances are made of."""
import numpy as np
import torch


def attend(q, k, v, seen, scale):
    """q [Hq, d], k/v [n, Hkv, d] (any dtype), seen bool [n] -> in float64
    out [Hq, d], weights [Hq, n], mix = sum p |v| [Hq, d] and
    reach = max over seen tokens of scale * sum |q k| [Hq].  Nothing seen:
    zeros."""
    q, k, v = q.double(), k.double(), v.double()
    Hq, d = q.shape
    n, Hkv = k.shape[0], k.shape[1]
    out = torch.zeros(Hq, d, dtype=torch.float64, device=q.device)
    mix, w = out.clone(), torch.zeros(Hq, n, dtype=torch.float64, device=q.device)
    reach = torch.zeros(Hq, dtype=torch.float64, device=q.device)
    idx = torch.nonzero(seen).flatten()
    if idx.numel() == 0:
        return out, w, mix, reach
    for h in range(Hq):
        kh, vh = k[idx, h // (Hq // Hkv)], v[idx, h // (Hq // Hkv)]
        p = torch.softmax((kh @ q[h]) * scale, 0)
        w[h, idx] = p
        out[h], mix[h] = p @ vh, p @ vh.abs()
        reach[h] = (kh.abs() @ q[h].abs()).max() * abs(scale)
    return out, w, mix, reach


def window_seen(n, pos, window, sinks, device="cuda"):
    """Tokens of [0, n) that a query at position pos sees."""
    t = torch.arange(n, device=device)
    ok = t <= pos
    if window > 0:
        ok &= (t < sinks) | (t > pos - window)
    return ok


def logit_slack(reach, d):
    """Bound on a logit's error in fp32: products of 16-bit values are exact,
    and each of the d / 16 accumulation steps (and the alignment inside one)
    is off by at most two units of 2^-23 of the sum of the magnitudes; twice
    that for the scale's product and the exponential's argument."""
    return (2 * d / 16 + 4) * 2.0 ** -23 * reach


def out_bound(out, mix, reach, d, p_eps, out_eps, extra=0.0):
    """Elementwise bound on |output - out|: every weight is off by p_eps
    (its rounding) and by the logits' error (on both sides of the division),
    the output by out_eps."""
    w = p_eps + 2 * logit_slack(reach, d)[:, None] + 2.0 ** -19
    return w * mix + out_eps * (out.abs() + w * mix) + extra + 1e-30


HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def assert_within(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    over = err > bound
    if over.any():
        i = torch.nonzero(over)[0].tolist()
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} outside; first {i}: "
                             f"{float(err[tuple(i)]):.3e} > {float(bound[tuple(i)]):.3e}")


# ------------------------------------------------------------ the 4-bit format

def kv4_values(x, by):
    """fp32 values that rows x (numpy float32 [..., d]) stand for after the
    4-bit write with tensor scale `by`: the definition's fp32 operations."""
    with np.errstate(over="ignore"):
        y = (x.astype(np.float32) / np.float32(by)).astype(np.float32)
    y = np.clip(y, np.float32(-65504), np.float32(65504)).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore", divide="ignore"):
        zero = y.min(-1, keepdims=True).astype(np.float16).astype(np.float32)
        step = (np.maximum(y.max(-1, keepdims=True) - zero, np.float32(0)) / np.float32(15)).astype(np.float16)
        step = step.astype(np.float32)
        code = np.where(step > 0, np.clip(np.rint((y - zero) / step), 0, 15), np.float32(0)).astype(np.float32)
    bad = np.isnan(y).any(-1, keepdims=True)
    val = np.where(bad, np.float32(np.nan), zero + step * code)
    with np.errstate(over="ignore"):
        return (val * np.float32(by)).astype(np.float32).reshape(x.shape)


def kv4_block(cache, block, head, bs, d, value):
    """float64 [bs, d] of one head of one block of a 4-bit cache (numpy
    uint8 [NB, Hkv, bytes]), element by element by the documented places."""
    raw = np.ascontiguousarray(cache[block, head])
    words, half, G = raw[:bs * d // 2].view("<u4"), raw[bs * d // 2:].view("<f2").astype(np.float64), d // 32
    t, e = np.meshgrid(np.arange(bs), np.arange(d), indexing="ij")
    if value:
        w = ((t // 8 * 8 + e % 32 // 4) * 4 + t // 2 % 4) * G + e // 32
        c, par = 4 * (t % 2) + e % 4, (t // 2 * G + e // 32) * 2 + t % 2
    else:
        w, c, par = (4 * t + e % 32 // 8) * G + e // 32, e % 8, t * G + e // 32
    code = (words[w] >> (4 * c).astype(np.uint32)) & 15
    return half[par] * code + half[par + bs * G]
