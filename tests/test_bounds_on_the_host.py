"""What the host makes of bounds that lie far above the lengths."""
import paged_kv_cache_44_gb300 as pkv

MOST = 2 ** 31 - 1


def test_prompt_workspace_of_loose_bounds():
    f = pkv.prompt_workspace_size
    # few rows over many keys are split, whatever the bound: about as many partitions as for 32,768 keys
    near = f(2, 14, 9, 32768, 12, 2, 128)
    assert near > 1 << 20
    for bound in (1 << 24, 1 << 30, MOST - 128, MOST - 127, MOST):
        assert near // 2 <= f(2, 14, 9, bound, 12, 2, 128) <= 4 * near
        assert near // 2 <= f(2, 14, 9, bound, 12, 2, 128, bound, 0) <= 4 * near
        assert f(2, 14, 9, bound, 12, 2, 128, 100, 2) == 256
    # no more queries than there are
    for bound in (14, 65, 1 << 20, MOST - 254, MOST):
        assert f(2, 14, bound, 32768, 12, 2, 128) == f(2, 14, 14, 32768, 12, 2, 128)
    # partitions that the caller asks for: 2^24 of 128 keys for each of the 14 * 12 rows, in 64 bits
    rows = 14 * 12 * (1 << 24)
    assert 0 <= f(2, 14, 9, MOST, 12, 2, 128, partition_size=128) - 256 - rows * 130 * 4 < 1024
