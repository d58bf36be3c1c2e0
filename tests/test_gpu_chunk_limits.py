"""Chunk attention, the append and the page calls where a call is at an end of its
range: nothing to do, a page of the context that is missing."""

import pytest
import torch

from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib
from tests.test_gpu_chunk import Case
from tests.test_gpu_pages import DevicePool, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_lib()


# ------------------------------------------------------------- nothing to do

@pytest.mark.parametrize("layers", [0, 1, 3])
def test_append_of_no_tokens_still_writes_the_lengths(layers):
    shape = (layers,) if layers else ()
    kc = torch.ones((*shape, 4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    k = torch.empty((*shape, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    lens, after = dev([5, 0, 30]), dev([-1, -1, -1])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.sv_kv_append(k, k, kc, vc, dev([[0, 1], [2, -1], [3, 0]]), lens, dev([0, 0, 0, 0]), new_ctx_lens=after, workspace=ws)
    assert sv.sv_get_device_error(ws) == 0 and after.tolist() == [5, 0, 30]
    assert (kc == 1).all() and (vc == 1).all()


def test_attention_of_no_tokens():
    c = Case([20, 3], [1, 1], 8, 2, 64)
    q = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((0, 8), dtype=torch.float32, device="cuda")
    for most in (0, 4):
        assert c.run(q=q, out=torch.empty_like(q), lse=lse, cu_tokens=dev([0, 0, 0]), max_tokens=most) == 0


def test_copy_of_an_empty_list():
    k = torch.randn((2, 5, 2, 16, 64), device="cuda").to(torch.bfloat16)
    want, none = k.clone(), dev([])
    sv.sv_pages_copy(k, None, none, none, dev([3]))
    assert torch.equal(k, want)


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
