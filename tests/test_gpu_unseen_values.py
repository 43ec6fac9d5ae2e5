"""Values of K and V that no query sees, in the calls whose products run over
whole stages of 128 keys: a weight of 0 times what is not finite is not 0, so
these tests hold NaN and infinities wherever nothing may be read into a
result, and rows that see nothing beside rows that do."""
import pytest
import torch

from tests.test_gpu_prompt import call, inputs
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("part", [0, 128])
@pytest.mark.parametrize("bad", BAD)
def test_padding_of_length_0_behind_shared_blocks(part, bad):
    """A padding row is zeros whatever the tokens of its group hold, and a member that ends partitions before."""
    c = Case([(1024, [1100, 0, 1030, 200])], 12, 2, 128, 16, seed=22)
    want = c.run(128)
    at = c.tables[0, 900 // 16]
    c.vc[at] = bad                                       # seen by the members of 1,100 and 1,030
    out = c.run(part)
    assert (out[1] == 0).all()
    assert not torch.isfinite(out[0]).all()
    if part == 128:
        assert torch.equal(out[3], want[3])


@pytest.mark.parametrize("ql,kl", [([300, 40], [100, 10]), ([40, 20, 64], [10, 3, 1]), ([700], [129])])
@pytest.mark.parametrize("shape", [(4, 2, 64), (12, 2, 128), (3, 3, 128)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("part", [0, 128])
def test_prompt_rows_that_see_nothing(ql, kl, shape, part):
    q, k, v = inputs(ql, kl, *shape, seed=24)
    for bad in BAD:
        v2 = v.clone()
        v2[:] = bad
        out = call(q, k, v2, ql, kl, part=part)
        at = 0
        for a, b in zip(ql, kl):
            assert (out[at:at + a - b] == 0).all()
            assert not torch.isfinite(out[at + a - b:at + a]).any()
            at += a
