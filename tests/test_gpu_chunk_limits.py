"""Chunk attention, the append and the page calls where a call or its numbers are
at an end of their range: nothing to do (or nothing yet, in a captured step), tables
far wider than their sequences, a wrong sequence among others, weights at the lower
end of fp16, a page of the context that is missing, two streams at once.

Tolerance, as derived in test_gpu_chunk.py: eps / 2 (A + |out|) + 2e-4 A with
A = sum p |v| / l.  fp16 adds what its subnormal steps cost: weights are held as
p 2^7 against a running maximum, so one below 2^-21 is off by at most 2^-25 2^-7 =
2^-32, n of them by n 2^-32 max |v|; and an output below 2^-14 is rounded to a
multiple of 2^-24, off by 2^-25 at most.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib
from tests.test_gpu_chunk import Case
from tests.test_gpu_pages import DevicePool, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_lib()


def compare(c, rows=None, sm_scale=None):
    """The rows of the mask (all) against the float64 oracle, lse too; the others
    as they were (7)."""
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    q, k, v, table = f(c.q), np.nan_to_num(f(c.k)), np.nan_to_num(f(c.v)), c.table.cpu().numpy()
    kw = dict(window=c.window, sink=c.sink, sm_scale=sm_scale)
    want, lse = oracle.chunk_attention(q, k, v, table, c.ctx, c.cu_np, **kw)
    mean, _ = oracle.chunk_attention(q, k, np.abs(v), table, c.ctx, c.cu_np, **kw)
    got, got_lse = f(c.out), c.lse.cpu().numpy()
    rows = np.ones(c.T, dtype=bool) if rows is None else rows
    half = torch.finfo(c.dtype).eps / 2
    tol = half * (mean + np.abs(want)) * 1.001 + 2e-4 * mean
    if c.dtype == torch.float16:
        keys = max(a + b for a, b in zip(c.ctx, c.new))
        tol += keys * 2.0 ** -32 * np.abs(v).max() + 2.0 ** -25
    else:
        tol += torch.finfo(c.dtype).tiny
    worst = (np.abs(got[:c.T] - want)[rows] / tol[rows]).max()
    assert worst <= 1.0, worst
    assert np.abs(got_lse[:c.T] - lse)[rows].max() <= 1e-4
    assert (got[:c.T][~rows] == 7.0).all() and (got_lse[:c.T][~rows] == 7.0).all()


# ------------------------------------------------------------------ numbers

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,Hq,Hkv", [
    ([600], [1], 8, 2), ([3000], [1], 8, 2), ([900, 3000, 40], [1, 1, 1], 16, 1), ([3000], [5], 4, 1),   # the row kernel
    ([3000], [40], 8, 2), ([700, 2500], [300, 64], 4, 4), ([2000, 900], [33, 1], 8, 2),                  # and the tile kernel
])
def test_weights_below_the_least_fp16_number(ctx, new, Hq, Hkv, D):
    """One key outweighs the others by 2^25.05 and brings no value of its own: the
    output is what the others bring, each below half of fp16's least step."""
    c = Case(ctx, new, Hq, Hkv, D, "fp16", seed=31)
    c.q.zero_()
    c.q[..., 0] = 1
    c.k = torch.where(torch.isnan(c.k), c.k, torch.zeros_like(c.k))
    c.v.abs_()
    first = c.table[:, 0].long()
    c.k[first, :, 0, 0] = 1
    c.v[first, :, 0] = 0
    scale = 25.05 * math.log(2)
    assert c.run(sm_scale=scale) == 0
    compare(c, sm_scale=scale)


@pytest.mark.parametrize("new", [[1], [40]])
def test_weights_over_the_whole_range_of_fp16(new):
    c = Case([4000], new, 8, 2, 64, "fp16", seed=32)
    c.q.mul_(2.0)  # scores over about +- 8 standard deviations of 2: weights from 1 to 2^-30
    assert c.run() == 0
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    k, v = np.nan_to_num(f(c.k)), np.nan_to_num(f(c.v))
    want, lse = oracle.chunk_attention(f(c.q), k, v, c.table.cpu().numpy(), c.ctx, c.cu_np)
    mean, _ = oracle.chunk_attention(f(c.q), k, np.abs(v), c.table.cpu().numpy(), c.ctx, c.cu_np)
    # scores are twice those of the derivation above: their 32-bit error too
    tol = 2.0 ** -11 * (mean + np.abs(want)) * 1.001 + 4e-4 * mean + 4100 * 2.0 ** -32 * np.abs(v).max() + 2.0 ** -25
    assert (np.abs(f(c.out) - want) <= tol).all() and np.abs(c.lse.cpu().numpy() - lse).max() <= 2e-4


# ------------------------------------------------------------------ tables

@pytest.mark.parametrize("width", [300, 2048])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,window,sink", [
    ([511], [1], 8, 2, 64, "bf16", 0, 0), ([1000, 0, 37, 1600] * 4, [1] * 16, 32, 8, 128, "bf16", 0, 0),
    ([500] * 4, [100, 33, 200, 17], 16, 4, 64, "fp16", 0, 0), ([0] * 3, [1024, 300, 1], 8, 2, 128, "bf16", 0, 0),
    ([700, 40, 1300, 9], [7, 1, 8, 300], 8, 2, 64, "bf16", 0, 0), ([900, 3000], [1, 120], 8, 2, 128, "fp16", 500, 20),
])
def test_tables_far_wider_than_their_sequences(ctx, new, Hq, Hkv, D, dtype, window, sink, width):
    """An engine's table has one width whatever its sequences hold; entries behind
    them are -1."""
    c = Case(ctx, new, Hq, Hkv, D, dtype, window=window, sink=sink, seed=width + len(ctx))
    wide = torch.full((c.B, width), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    assert c.run() == 0
    compare(c)


@pytest.mark.parametrize("batch,longest,new", [(3, 10, 1), (3, 900, 1), (50, 900, 1), (400, 100, 1), (3, 9000, 1),
                                               (5, 2000, 40), (70, 700, 20)])
def test_a_wrong_length_leaves_the_others_right(batch, longest, new):
    """The work is shared out anew without the sequence: the others' rows are
    compared with the oracle, element by element, and their lse."""
    rng = np.random.default_rng(batch + longest)
    ctx = rng.integers(0, longest, batch).tolist()
    ctx[1] = longest
    news = [new] + [1 if i % 2 else new for i in range(1, batch)]
    c = Case(ctx, news, 16, 4, 64, "bf16", seed=longest)
    assert c.run() == 0
    compare(c)
    for at in (0, batch // 2, batch - 1):
        for bad in (100000, -1):
            c.lens[at] = bad
            c.out.fill_(7.0)
            c.lse.fill_(7.0)
            assert c.run() == sv.SV_DEVERR_BAD_LENGTH
            rows = np.ones(c.T, dtype=bool)
            rows[c.cu_np[at]:c.cu_np[at + 1]] = False
            compare(c, rows)
        c.lens[at] = ctx[at]


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


# ------------------------------------------------------------------- steps

@pytest.mark.parametrize("batch,Hq,Hkv,width,most", [
    (1, 8, 2, 100, 1), (3, 8, 2, 20, 1), (3, 8, 2, 2, 1), (40, 16, 4, 300, 1),     # the row kernel's ways of sharing
    (1, 8, 2, 100, 300), (4, 32, 8, 300, 200), (40, 16, 4, 20, 64), (2, 64, 2, 50, 1),  # the tile kernel, both, and cut units
])
def test_a_step_in_which_no_sequence_brings_a_token(batch, Hq, Hkv, width, most):
    """A captured step of fixed size: all its rows are padding, later they are not."""
    c = Case([min(5 + i, width * 16 - most) for i in range(batch)], [1] * batch, Hq, Hkv, 64, seed=batch)
    c.table = torch.cat([c.table, torch.full((batch, width), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    p = c.params(max_tokens=most)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_chunk_attention(p)
    cu = c.cu.clone()
    for _ in range(2):
        c.cu.zero_()
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        graph.replay()
        assert sv.sv_get_device_error(c.ws) == 0 and (c.out == 7.0).all() and (c.lse == 7.0).all()
        c.cu.copy_(cu)
        graph.replay()
        assert sv.sv_get_device_error(c.ws) == 0
        compare(c)


def test_two_streams_at_once():
    """Calls of every kind on two streams, each with its own workspace and pages."""
    steps = [[Case([900, 3, 200], [70, 1, 1], 32, 8, 128, "fp16", seed=41), Case([3000, 40], [1, 1], 8, 2, 64, seed=42)],
             [Case([0, 700], [300, 1], 8, 2, 128, seed=43), Case([500] * 30, [1] * 30, 16, 4, 64, "fp16", seed=44)]]
    params = [[c.params() for c in cases] for cases in steps]
    pools = [DevicePool(3, 8, 40), DevicePool(40, 8, 1100)]
    news = [dev([33] * 3), dev([20] * 40)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, calls, d, new in zip(streams, params, pools, news):
            with torch.cuda.stream(s):
                for p in calls:
                    sv.sv_chunk_attention(p)
                sv.sv_pages_reserve(d.ctx, new, d.table, d.held, d.refs, d.src, d.dst, d.count, workspace=d.ws)
                sv.sv_pages_copy(d.k, d.v, d.src, d.dst, d.count, workspace=d.ws)
                sv.sv_pages_release(d.ctx, d.table, d.held, d.refs, workspace=d.ws)
    for s, calls, d, new in zip(streams, params, pools, news):
        with torch.cuda.stream(s):
            sv.sv_pages_reserve(d.ctx, new, d.table, d.held, d.refs, d.src, d.dst, d.count, workspace=d.ws)
    torch.cuda.synchronize()
    for cases in steps:
        for c in cases:
            assert sv.sv_get_device_error(c.ws) == 0
            compare(c)
    for d, new in zip(pools, news):
        assert d.error() == 0 and d.model.reserve(new.tolist()) == []
        d.same()
