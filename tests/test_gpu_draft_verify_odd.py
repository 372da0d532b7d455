"""draft_verify where draft entries are no probabilities: they weigh what the rule says, however the sums are taken."""
import numpy as np
import pytest
import torch

from tests.test_gpu_draft_verify import Case

pytestmark = pytest.mark.gpu


def odd(t, which, seed):
    """Every few entries of the rows are replaced."""
    r = np.random.RandomState(seed)
    V = t.shape[-1]
    for value in which:
        t[..., torch.from_numpy(r.permutation(V)[:max(1, V // 9)]).cuda()] = value


@pytest.mark.parametrize("kind", ["rows", "distinct"])
@pytest.mark.parametrize("which", [[float("nan")], [-0.001, -7.0], [-0.0], [float("inf")], [-float("inf")], [2.5, 1e30],
                                   [float("nan"), -0.3, float("inf"), -1e-30, 1e-40]])
@pytest.mark.parametrize("rejected", [1, 2, 5])
@pytest.mark.parametrize("V", [40, 4099, 70001])
def test_odd_draft_entries(kind, which, rejected, V):
    """`rejected` children of the root and no other, most of them rejected: the next token is drawn from what they leave, by
    one quick pass (one rejected) or a general one."""
    c = Case(8, rejected + 1, V, kind, 1, near=2.0, seed=V + rejected)
    c.parent[:, 1:] = 0
    c.tokens[:, 1:] = torch.rand(8, V, device="cuda").argsort(-1)[:, :rejected].to(torch.int32)
    # what a child's token is proposed with is a probability, far above the target's
    c.draft, c.target = c.draft.contiguous(), c.target.contiguous()
    odd(c.draft, which, V)
    for b in range(8):
        c.draft[b, 0, c.tokens[b, 1:].long()] = 0.1
    c.u.fill_(0.99)
    c.call()
    c.check()
    assert (c.len == 1).any(), "no child was rejected"


@pytest.mark.parametrize("which", [[float("nan")], [-0.2], [float("nan"), -1.0, float("inf")]])
def test_odd_proposals(which):
    """The children's own entries too."""
    for kind in ("rows", "distinct"):
        c = Case(8, 9, 300, kind, 3, near=2.0, seed=4)
        c.draft = c.draft.contiguous()
        odd(c.draft, which, 5)
        c.u.fill_(0.9)
        c.call()
        c.check()


@pytest.mark.parametrize("which", [[float("nan")], [-0.001], [float("nan"), -0.3, -1e-30, 1e-40, 3.0, 400.0]])
@pytest.mark.parametrize("kind", ["rows", "distinct", "certain"])
def test_odd_target_entries(which, kind):
    """(At most 400 each and few: sums stay below 2^63 / 2^53.)"""
    c = Case(8, 4, 12 if 400.0 in which else 5000, kind, 2, near=2.0, seed=6)
    c.target = c.target.contiguous()
    odd(c.target, which, 7)
    c.u.fill_(0.9)
    c.call()
    c.check()
