"""Values of K and V that no query sees, in the calls whose products run over
whole stages of 128 keys: a weight of 0 times what is not finite is not 0, so
these tests hold NaN and infinities wherever nothing may be read into a
result, and rows that see nothing beside rows that do."""
import pytest
import torch

from tests.test_gpu_prompt import call, check, inputs
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), float("-inf")]


def hide(c, bad):
    """Put `bad` in every slot of c's pools that no sequence sees."""
    bs = c.bs
    seen = torch.zeros(c.kc.shape[0], bs, dtype=torch.bool)
    tab = c.tables.cpu()
    for s, n in enumerate(c.lens):
        for b in range(-(-n // bs)):
            seen[tab[s, b], :min(bs, n - b * bs)] = True
    for pool in (c.kc, c.vc):
        pool[~seen.cuda()] = bad


# members that all end inside the shared tokens: past the longest one its blocks have never been written
SHORT = [(512, [300, 17, 0, 1]), (256, [0, 0]), (128, [100, 127]), (640, [5, 600, 630]), (1024, [129, 128, 0]),
         (2048, [40]), (64, [100, 20])]


@pytest.mark.parametrize("shape", [(4, 2, 64, 16), (12, 2, 128, 16), (28, 4, 128, 32), (3, 3, 128, 16), (64, 1, 64, 32)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("part", [0, -1, 128])
@pytest.mark.parametrize("bad", BAD)
def test_shared_blocks_past_every_member(shape, part, bad):
    c = Case(SHORT, *shape, seed=21, before=[3], after=[0, 50])
    hide(c, bad)
    out = c.run(part)
    c.check(out)
    for s, n in enumerate(c.lens):
        if n == 0:
            assert (out[s] == 0).all()


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


@pytest.mark.parametrize("part", [0, 128])
@pytest.mark.parametrize("bad", BAD)
def test_tokens_that_only_longer_members_see(part, bad):
    """Values that are not finite reach the members that see them, as in a decode, and no others."""
    c = Case([(1024, [1100, 640, 1023, 1024, 650])], 12, 2, 128, 16, seed=26)
    want = c.run(part)
    c.check(want)
    c.vc[c.tables[0, 1008 // 16], 15] = bad              # token 1,023
    c.vc[c.tables[0, 640 // 16], 9] = bad                # token 649
    out = c.run(part)
    assert torch.equal(out[1], want[1])
    assert not any(torch.isfinite(out[s]).any() for s in (0, 2, 3, 4))


def test_a_large_group_with_short_members():
    c = Case([(1536, [(37 * i) % 1100 for i in range(90)] + [1333]), (256, [256] * 40 + [300])], 8, 2, 128, 16, seed=23)
    hide(c, float("nan"))
    for part in (0, 256):
        c.check(c.run(part))


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


@pytest.mark.parametrize("shape", [(4, 2, 64), (12, 2, 128), (28, 4, 128), (3, 3, 64)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 3), (128, 128), (257, 130), (1000, 0)])
@pytest.mark.parametrize("part", [0, 128, -1])
@pytest.mark.parametrize("few", [True, False], ids=["few", "many"])
def test_prompt_keys_behind_every_window(shape, window, sinks, part, few):
    """Keys between the sinks and the first query's window: no query of the sequence sees them."""
    ql, kl = ([5, 64, 1, 9], [2000, 700, 130, 9]) if few else ([5, 130, 300, 257], [2000, 1031, 777, 257])
    q, k, v = inputs(ql, kl, *shape, seed=25)
    clean = call(q, k, v, ql, kl, True, window, sinks, part=part)
    check(clean, q, k, v, ql, kl, True, window, sinks, shape[2] ** -0.5)
    for bad in BAD:
        k2, v2, at = k.clone(), v.clone(), 0
        for a, b in zip(ql, kl):
            lo, hi = sinks, b - a - window + 1
            if hi > lo:
                k2[at + lo:at + hi], v2[at + lo:at + hi] = bad, bad
            at += b
        assert torch.equal(call(q, k2, v2, ql, kl, True, window, sinks, part=part), clean)
