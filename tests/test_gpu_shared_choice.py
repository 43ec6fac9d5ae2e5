"""The automatic choice of the shared decode where groups differ in size, and
with sequences that share nothing among them or as a group of their own."""
import pytest
import torch

from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu


def test_one_large_group_among_small_ones():
    """No more than all sequences can read the shared tokens again, however many groups there are."""
    groups = [(304, [305 + i for i in range(100)])] + [(16 * (1 + i % 5), [100, 90 + i]) for i in range(50)]
    c = Case(groups + [(0, [700, 1, 0, 33])], 12, 2, 128, 16, seed=51)
    out = c.run(sharing="auto")
    c.check(out)
    c.check(c.run())
    c.starts.fill_(-1)                                    # the groups are not looked at
    assert torch.equal(c.run(sharing="auto"), out)


@pytest.mark.parametrize("among", [False, True])
def test_groups_that_share_nothing(among):
    """Sequences that share nothing as a group between or behind the others, or in no group: one result."""
    big = [(2048, [2049 + 7 * i for i in range(40)]), (2048, [2048] * 40)]
    alone = (0, [5, 900, 0, 2500])
    c = Case(big[:1] + [alone] + big[1:] if among else big + [alone], 4, 4, 128, 16, seed=52)
    for sharing in ("auto", "always"):
        c.check(c.run(sharing=sharing))
    if not among:
        c.starts, c.shared = c.starts[:3].contiguous(), c.shared[:2].contiguous()
        c.check(c.run())
