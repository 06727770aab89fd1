"""idx_logit_probs with penalties for the tokens of drafted trees alone: neither counts nor biases.

Tolerances are those of the tests of idx_logit_probs.
"""

import pytest
import torch
from test_gpu_probs import Case

pytestmark = pytest.mark.gpu


def trees(sizes, seed):
    """Masks of each node's ancestors and itself, in trees whose nodes have parents drawn at random among those before."""
    g = torch.Generator().manual_seed(seed)
    masks = []
    for n in sizes:
        own = []
        for i in range(n):
            up = own[int(torch.randint(0, i, (1,), generator=g))] if i > 0 else 0
            own.append(up | 1 << i)
        masks += own
    signed = [m - 2**64 if m >> 63 else m for m in masks]
    return torch.tensor(signed, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("sizes", [[64] * 30, [33, 64, 1, 40, 8, 50, 64, 34] * 6, [64], [5] * 200])
def test_trees_without_counts(lib, sizes):
    """More rows than run at once, so that CTAs begin inside requests and go on to others; the same to the bit each time."""
    cu = [0]
    for n in sizes:
        cu.append(cu[-1] + n)
    c = Case(cu, 300, tree=trees([*sizes, 1], len(sizes)), pad=1)  # a row behind the last request
    del c.args["counts"]
    c.check(lib)
    first = c.probs.clone()
    for _ in range(5):
        c.probs.fill_(9.0)
        assert torch.equal(c.run(lib).probs[:, :300], first[:, :300])


def test_chains_of_masks_without_counts(lib):
    """A tree that is a chain gives what no mask gives."""
    sizes = [64, 37, 64]
    tree = torch.cat([torch.tensor([(1 << i + 1) - 1 if i < 63 else -1 for i in range(n)], dtype=torch.int64) for n in sizes]).cuda()
    c = Case([0, 64, 101, 165], 2000, tree=tree)
    del c.args["counts"]
    c.check(lib)
    want = c.probs.clone()
    del c.args["tree_mask"]
    assert torch.equal(c.run(lib).probs, want)
