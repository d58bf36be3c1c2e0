"""Chunk attention, the append and the page calls where a call is at an end of its
range: a page of the context that is missing."""

import pytest
import torch

from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib
from tests.test_gpu_pages import DevicePool, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_lib()


# ------------------------------------------------------------------- pages

@pytest.mark.parametrize("rows", [3, 40])  # (one CTA, a cluster)
def test_reserve_wants_the_pages_of_the_context(rows):
    """A row whose last context page is not held (a rollback that left ctx_lens as
    it was) takes no part: the page would come back without its tokens."""
    d = DevicePool(rows, 6, 64)
    start = [20] + [16] * (rows - 1)
    assert d.reserve(start) == d.model.reserve(start) == []
    d.set_ctx(start)
    keep = [16] * rows
    sv.sv_pages_release(dev(keep), d.table, d.held, d.refs, workspace=d.ws)
    d.model.release(keep)
    d.same()
    for length in (17, 20, 31):
        d.set_ctx([length] + start[1:])
        before = [t.clone() for t in (d.table, d.held, d.refs)]
        assert d.reserve([40] + start[1:]) == [] and d.error() == sv.SV_DEVERR_BAD_LENGTH
        assert all(torch.equal(a, b) for a, b in zip(before, (d.table, d.held, d.refs)))
    # the others are served all the same, and the row once its length says what it holds
    new = [40] + [16] * (rows - 2) + [33]
    d.reserve(new)
    assert d.error() == sv.SV_DEVERR_BAD_LENGTH
    d.model.ctx[0] = 40  # (no growth: the row stays out of the model's call)
    assert d.model.reserve(new) == []
    d.model.ctx[0] = length
    d.same()
    d.set_ctx([16] + start[1:-1] + [33])
    assert d.reserve([40] + [0] * (rows - 1)) == d.model.reserve([40] + [0] * (rows - 1)) == [] and d.error() == 0
    d.same()
