"""What the host makes of bounds that lie far above the lengths, and of groups
whose bounds allow more members than there are sequences."""
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


def test_no_more_members_than_sequences():
    """The estimate of what is read again counts at most the sequences there are."""
    f = pkv.shared_workspace_size
    shape = (200, 51, 64, 8, 128, 16, 33792)
    plain = pkv.decode_workspace_size(200, 64, 8, 128, 16, 33792)
    # 199 sequences behind the first of their group, 304 tokens of 8 heads: 236 MiB; 51 groups of 100 would be 6 GiB
    for members in (100, 65535):
        assert f(*shape, 304, members) == plain < f(*shape, 304, members, sharing="always")
        assert f(*shape, 512, members) == f(*shape, 512, members, sharing="always")       # 398 MiB
    # what bounds it below the sequences is still the groups' bound
    assert f(*shape, 2048, 2) == f(*shape, 2048, 2, sharing="always")                     # 51 * 16 MiB
    assert f(200, 1, *shape[2:], 2048, 2) == plain
