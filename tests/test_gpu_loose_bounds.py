"""Bounds of the lengths that are far above them, as a caller passes who has
one constant for every step."""
import pytest
import torch

from tests.test_gpu_prompt import BF, inputs, check, starts

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_cache_44_gb300 as pkv

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("shape", [(12, 2, 128), (3, 3, 64)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ql,kl", [([300, 1, 129], [300, 1, 129]), ([5, 9], [4000, 9000]), ([200, 30], [100, 500])])
@pytest.mark.parametrize("bound_q,bound_k", [(MOST, MOST), (MOST - 254, MOST - 128), (1 << 30, 1 << 30), (100000, 100000)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 4)])
def test_prompt(shape, ql, kl, bound_q, bound_k, window, sinks):
    q, k, v = inputs(ql, kl, *shape, seed=31)
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # the call's own workspace, one of the size that the bounds ask for, the smallest one
    Hq, Hkv, d = shape
    own = pkv.make_prompt_workspace(len(ql), sum(ql), bound_q, bound_k, Hq, Hkv, d, window, sinks)
    assert own.numel() < 1 << 30
    for ws in (None, own, torch.zeros(256, dtype=torch.uint8, device="cuda")):
        out.fill_(7.0)
        pkv.prompt_attention(out, q, k, v, starts(ql), bound_q, d ** -0.5, key_start=starts(kl), max_key_len=bound_k,
                             window=window, num_sinks=sinks, workspace=ws, err_word=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        check(out, q, k, v, ql, kl, True, window, sinks, d ** -0.5)


@pytest.mark.parametrize("window", [0, 150])
def test_prompt_in_partitions(window):
    """Partitions that the caller asks for take a workspace by the keys there are, not by the bound."""
    ql, kl = [5, 9], [1000, 3000]
    q, k, v = inputs(ql, kl, 12, 2, 128, seed=32)
    out = torch.zeros(q.shape, dtype=BF, device="cuda")
    pkv.prompt_attention(out, q, k, v, starts(ql), MOST, 128 ** -0.5, key_start=starts(kl), max_key_len=MOST, window=window,
                         partition_size=128)
    check(out, q, k, v, ql, kl, True, window, 0, 128 ** -0.5)
