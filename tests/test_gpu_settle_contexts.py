"""idx_settle_drafts where there is nothing to move: contexts and counts alone."""

import pytest
import torch
from test_gpu_pages import Settle, dev, np_

from oracle import serve

pytestmark = pytest.mark.gpu
PATHS = [[2, 4], [3, 5], [1, 2, 3], [5]]  # nodes at their places, and others


def settle():
    return Settle([6, 6, 6, 6], paths=PATHS)


def test_without_caches_no_node_has_a_place(lib):
    s = settle()
    s.caches = []
    s.check(lib)


@pytest.mark.parametrize("shape", [(0, 8, 16, 4), (2, 0, 16, 4), (2, 8, 16, 0)])
def test_caches_of_nothing(lib, shape):
    s = settle()
    s.caches = [torch.zeros(shape, device="cuda")]
    s.check(lib)


def test_nodes_are_looked_at_all_the_same(lib):
    s = settle()
    s.caches, s.nodes[1, 1] = [], 1  # before its place
    s.check(lib, status=lib.ST_BAD_TREE)


def test_without_slots(lib):
    """The C entry takes no slots where there are no caches."""
    s = settle()
    _, ctx, counts = serve.settle([], s.slots, s.cu, s.tokens, s.nodes, s.accepted, s.ctx, s.counts)
    cu, tokens, nodes, accepted, ctx_in, counted, status = (dev(x) for x in (s.cu, s.tokens, s.nodes, s.accepted, s.ctx, s.counts, [0]))
    out = torch.zeros_like(ctx_in)
    rc = lib.load_library().idx_settle_drafts(None, 0, 0, 16, None, cu.data_ptr(), 4, 24, tokens.data_ptr(), nodes.data_ptr(), s.max_out, accepted.data_ptr(),
                                              ctx_in.data_ptr(), out.data_ptr(), counted.data_ptr(), counted.stride(0), counted.shape[1], status.data_ptr(),
                                              torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and status.item() == 0
    assert (np_(out) == ctx).all() and (np_(counted) == counts).all()
