"""A layer's way from prompts to decoding steps, as a server takes it: the
block manager's slots and tables, the rotary write, attention over the whole
prompt, query chunks behind a cached prefix, and steps of one token for
requests that share a system prompt.  Every stage is held against 64 bits."""
import numpy as np
import pytest
import torch

from tests import plain64 as P64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

BF = torch.bfloat16
BS = 16


def table(positions, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat((a.cos(), a.sin()), 1).float().cuda()


def turned(x, cs, pos, rot):
    """The rotation in 64 bits, and the size |a| + |b| of each value's pair."""
    x, half = x.double().clone(), rot // 2
    size = x.abs()
    c, s = cs[pos, None, :half].double(), cs[pos, None, half:].double()
    a, b = x[..., :half].clone(), x[..., half:rot].clone()
    x[..., :half], x[..., half:rot] = a * c - b * s, b * c + a * s
    size[..., :half] = size[..., half:rot] = a.abs() + b.abs()
    return x, size


def rounded_once(got, want, size):
    """bf16 of an fp32 rotation: half a step of bf16, and two products and a sum of fp32."""
    err = (got.double() - want).abs()
    slack = 3 * 2.0 ** -24 * size
    assert (err <= 2.0 ** -8 * (want.abs() + slack) + slack).all()


@pytest.mark.parametrize("Hq,Hkv,d,rot", [(12, 2, 128, 128), (4, 4, 64, 32)])
def test_a_layer(Hq, Hkv, d, rot):
    g = torch.Generator(device="cuda").manual_seed(1)
    system, own, steps = 100, [37, 1, 64, 150, 20], 4
    S, far = len(own), 400
    cs = table(far, rot)
    scale = d ** -0.5
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = pkv.BlockPool(120, BS)
    kc, vc = (torch.full((120, BS, Hkv, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    # what the projections leave, token by token: the system prompt's rows are everybody's
    head = torch.randn(system, Hq + 2 * Hkv, d, device="cuda", generator=g).to(BF)
    rows = [torch.cat((head, torch.randn(n + steps, Hq + 2 * Hkv, d, device="cuda", generator=g).to(BF))) for n in own]
    ids = [list(range(system)) + [1000 * (s + 1) + i for i in range(n)] for s, n in enumerate(own)]

    def attend(q, s, n, pos):
        """64-bit attention of q [Hq, d] at position pos to what the cache holds of sequence s."""
        tab = torch.from_numpy(pool.block_tables([s], 32)[0][0]).cuda().long()
        k, v = (c[tab].flatten(0, 1)[:n] for c in (kc, vc))
        seen = torch.arange(n, device="cuda") <= pos
        return P64.attend(q, k, v, seen, scale)

    def check(out, q, s, n, pos):
        o, _, mix, reach = attend(q, s, n, pos)
        P64.assert_within(out, o, P64.out_bound(o, mix, reach, d, 2.0 ** -8, 2.0 ** -8), f"request {s}, position {pos}")

    def write(x, pos, slots):
        """Rotary write of projected rows x; Q and K come back."""
        q, k, v = x.split([Hq, Hkv, Hkv], 1)
        q_out, k_out = torch.empty(len(x), Hq, d, dtype=BF, device="cuda"), torch.empty(len(x), Hkv, d, dtype=BF, device="cuda")
        pkv.rotary_kv_write(q, k, v, pos, cs, q_out, k_out, kc, vc, slots)
        for got, raw in ((q_out, q), (k_out, k)):
            rounded_once(got, *turned(raw, cs, pos, rot))
        at = slots.long()
        assert torch.equal(kc.view(-1, Hkv, d)[at], k_out) and torch.equal(vc.view(-1, Hkv, d)[at], v)
        return q_out, k_out, v

    # the first request computes its whole prompt; the others find the system prompt's blocks in the cache
    cached = [pool.add_sequence(s, ids[s]) for s in range(S)]
    assert cached[0] == 0 and all(c == system // BS * BS for c in cached[1:])
    for s in range(S):
        n, lo = system + own[s], cached[s]
        tab = pool.block_tables([s], 32)[0][0]
        pos = torch.arange(lo, n, device="cuda")
        slots = torch.from_numpy(tab.astype(np.int64)).cuda()[pos // BS] * BS + pos % BS
        q, k, v = write(rows[s][lo:n], pos, slots)
        out, start = torch.zeros_like(q), torch.tensor([0, n - lo], **i32)
        if lo == 0:
            pkv.prompt_attention(out, q, k, v, start, n, scale)
        else:
            t, lens = (torch.from_numpy(x).cuda() for x in pool.block_tables([s], 32))
            pkv.paged_attention_prefill(out, q, kc, vc, t, lens, start, n - lo, n, scale)
        for i in (0, (n - lo) // 2, n - lo - 1):
            check(out[i], q[i], s, n, lo + i)
    # the same prompt, its queries behind the cached part, over K and V that lie side by side
    q, k, v = rows[0][:system + own[0]].split([Hq, Hkv, Hkv], 1)
    n, tail = system + own[0], own[0]
    whole, part = torch.zeros(n, Hq, d, dtype=BF, device="cuda"), torch.zeros(tail, Hq, d, dtype=BF, device="cuda")
    pkv.prompt_attention(whole, q, k, v, torch.tensor([0, n], **i32), n, scale)
    pkv.prompt_attention(part, q[-tail:], k, v, torch.tensor([0, tail], **i32), tail, scale, key_start=torch.tensor([0, n], **i32),
                         max_key_len=n)
    for i in (0, tail - 1):
        o, _, mix, reach = P64.attend(q[n - tail + i], k, v, torch.arange(n, device="cuda") <= n - tail + i, scale)
        bound = P64.out_bound(o, mix, reach, d, 2.0 ** -8, 2.0 ** -8)
        P64.assert_within(part[i], o, bound)
        P64.assert_within(whole[n - tail + i], o, bound)

    # steps of one token each, recorded once: the buffers' contents change from step to step
    shared = system // BS * BS
    x = torch.empty(S, Hq + 2 * Hkv, d, dtype=BF, device="cuda")
    q_out, out = torch.empty(S, Hq, d, dtype=BF, device="cuda"), torch.empty(S, Hq, d, dtype=BF, device="cuda")
    pos, slots = torch.zeros(S, dtype=torch.int64, device="cuda"), torch.full((S,), -1, dtype=torch.int64, device="cuda")
    tabs, lens = torch.zeros(S, 32, **i32), torch.ones(S, **i32)
    groups, common = torch.tensor([0, S], **i32), torch.tensor([shared], **i32)
    bounds = (max(own) + system + steps, shared, S)
    ws = pkv.make_shared_workspace(S, 1, Hq, Hkv, d, BS, *bounds, sharing="always")

    def step():
        q, k, v = x.split([Hq, Hkv, Hkv], 1)
        pkv.rotary_kv_write(q, k, v, pos, cs, q_out, None, kc, vc, slots)
        pkv.paged_attention_decode_shared(out, q_out, kc, vc, tabs, lens, groups, common, *bounds, scale, workspace=ws,
                                          sharing="always")

    graph = None
    for i in range(steps):
        new, copies = pool.append_tokens(range(S), [5000 + 10 * s + i for s in range(S)])
        assert len(copies) == 0
        t, n = pool.block_tables(range(S), 32)
        tabs.copy_(torch.from_numpy(t)), lens.copy_(torch.from_numpy(n)), slots.copy_(torch.from_numpy(new))
        pos.copy_(lens - 1)
        for s in range(S):
            x[s] = rows[s][system + own[s] + i]
        if graph is None:
            step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay()
        torch.cuda.synchronize()
        want, size = turned(x[:, :Hq], cs, pos, rot)
        rounded_once(q_out, want, size)
        for s in range(S):
            check(out[s], q_out[s], s, int(n[s]), int(n[s]) - 1)
