"""Chunk attention and the K/V append through the binding, against the float64
oracle.

Tolerances, derived: out = sum p v / l.  Each p is rounded to the 16-bit type
before the second product (half a step, eps / 2, relative) and the output once
more, so |error| <= eps / 2 (A + |out|) with A = sum p |v| / l; scores, sums
and the exponential are 32-bit: 128 products of 16-bit values summed in any
order are off by at most 128 2^-24 sum |q k| scale, below 1e-4 for these
inputs (sum |q k| scale < 12), which is also the bound of lse; it moves out by
at most 2e-4 A.  Partial results of cut sequences are 32-bit (no further
rounding).
"""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_lib()


class Case:
    """Random chunk; slots no row may read hold NaN, ids no row may use are -1."""

    def __init__(self, ctx, new, Hq, Hkv, D, dtype="bf16", window=0, sink=0, seed=0, q_pad=0, extra_rows=0, extra_pages=3):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.window, self.sink, self.dtype = ctx, new, window, sink, DTYPES[dtype]
        self.B, self.Hq, self.Hkv, self.D = len(ctx), Hq, Hkv, D
        need = [-(-(c + n) // 16) for c, n in zip(ctx, new)]
        self.pages = sum(need) + extra_pages
        order = rng.permutation(self.pages)
        width = max(max(need), 1) + 1
        table = np.full((self.B, width), -1, dtype=np.int32)
        k = torch.full((self.pages, Hkv, 16, D), float("nan"))
        v = torch.full((self.pages, Hkv, 16, D), float("nan"))
        at = 0
        for b in range(self.B):
            for lp in range(need[b]):
                # a page that the window has left behind for every row is gone
                first = max(0, ctx[b] - window + 1) if window else 0
                lo, hi = lp * 16, min(lp * 16 + 16, ctx[b] + new[b])
                page = order[at]
                at += 1
                if window and hi <= first and lo >= sink:
                    continue
                table[b, lp] = page
                k[page, :, :hi - lo] = torch.randn((Hkv, hi - lo, D), generator=g)
                v[page, :, :hi - lo] = torch.randn((Hkv, hi - lo, D), generator=g)
        self.T = sum(new)
        rows = self.T + extra_rows
        wide = torch.randn((rows, Hq + q_pad, D), generator=g).to(self.dtype).cuda()
        self.q = wide[:, :Hq]
        self.k, self.v = k.to(self.dtype).cuda(), v.to(self.dtype).cuda()
        self.table = torch.from_numpy(table).cuda()
        self.cu_np = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.cu = torch.from_numpy(self.cu_np).cuda()
        self.lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.out = torch.full((rows, Hq + q_pad, D), 7.0, dtype=self.dtype, device="cuda")[:, :Hq]
        self.lse = torch.full((rows, Hq), 7.0, device="cuda")

    def params(self, **kw):
        kw = {**dict(q=self.q, k_cache=self.k, v_cache=self.v, block_table=self.table, ctx_lens=self.lens,
                     cu_tokens=self.cu, out=self.out, lse=self.lse, max_tokens=max(self.new),
                     window_tokens=self.window, sink_tokens=self.sink), **kw}
        p = sv.make_chunk_params(**kw)
        self.ws = torch.zeros(sv.sv_chunk_attention_workspace_size(p), dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = self.ws.data_ptr(), self.ws.numel()
        return p

    def run(self, **kw):
        p = self.params(**kw)
        sv.sv_chunk_attention(p)
        torch.cuda.synchronize()
        return sv.sv_get_device_error(self.ws)

    def check(self, sm_scale=None, rows=None):
        """Compares the first `rows` rows (all) and requires the others untouched."""
        f = lambda t: t.float().cpu().numpy()  # noqa: E731
        q, k, v, table = f(self.q), f(self.k), f(self.v), self.table.cpu().numpy()
        kw = dict(window=self.window, sink=self.sink, sm_scale=sm_scale)
        # masked positions may hold NaN: the oracle multiplies by zero weights, so clear what nobody sees
        k, v = np.nan_to_num(k), np.nan_to_num(v)
        want, lse = oracle.chunk_attention(q, k, v, table, self.ctx, self.cu_np, **kw)
        mean, _ = oracle.chunk_attention(q, k, np.abs(v), table, self.ctx, self.cu_np, **kw)
        got, got_lse = f(self.out), self.lse.cpu().numpy()
        rows = self.T if rows is None else rows
        own = slice(0, rows)
        half = torch.finfo(self.dtype).eps / 2
        tol = half * (mean + np.abs(want)) * 1.001 + 2e-4 * mean + torch.finfo(self.dtype).tiny
        worst = (np.abs(got[own] - want[own]) / tol[own]).max()
        assert worst <= 1.0, worst
        assert np.isfinite(got_lse[own]).all() and np.abs(got_lse[own] - lse[own]).max() <= 1e-4
        assert (got[rows:] == 7.0).all() and (got_lse[rows:] == 7.0).all()


HEADS = [(8, 2, 64), (4, 4, 128), (32, 8, 128), (6, 2, 64), (7, 1, 128), (16, 1, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("ctx,new", [
    ([0], [1]), ([1], [1]), ([15], [1]), ([16], [1]), ([511], [1]), ([1000, 0, 37, 1600, 16], [1, 1, 1, 1, 1]),
    ([100, 7, 0], [2, 1, 2]),
])
def test_single_tokens(Hq, Hkv, D, dtype, ctx, new):
    c = Case(ctx, new, Hq, Hkv, D, dtype, seed=len(ctx) + Hq)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS + [(3, 3, 64), (20, 1, 64), (128, 1, 128), (65, 1, 64)])
@pytest.mark.parametrize("ctx,new", [
    ([0], [17]), ([0], [128]), ([0], [129]), ([5], [300]), ([127, 0, 700, 33], [64, 1, 131, 7]),
    ([0, 240], [0, 257]), ([1023], [33]),
])
def test_chunks(Hq, Hkv, D, dtype, ctx, new):
    c = Case(ctx, new, Hq, Hkv, D, dtype, seed=sum(new) + Hq)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 64, "bf16"), (32, 8, 128, "fp16"), (5, 1, 128, "bf16")])
@pytest.mark.parametrize("window,sink", [(1, 0), (16, 0), (17, 5), (100, 64), (333, 1), (5000, 64), (128, 130)])
@pytest.mark.parametrize("ctx,new", [([900, 3], [1, 1]), ([900, 0, 31], [140, 70, 1]), ([0], [513])])
def test_windows(Hq, Hkv, D, dtype, window, sink, ctx, new):
    c = Case(ctx, new, Hq, Hkv, D, dtype, window=window, sink=sink, seed=window)
    assert c.run() == 0
    c.check()


def test_long_contexts_are_cut_between_workers():
    c = Case([20000, 3], [1, 1], 8, 2, 128, "fp16", seed=3)
    assert c.run() == 0
    c.check()
    c = Case([9000], [40], 8, 2, 128, "bf16", seed=4)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("width", [1, 2, 3, 32, 33, 64, 65, 256, 257])
@pytest.mark.parametrize("batch,Hq,Hkv", [(1, 8, 2), (40, 16, 4)])
def test_widths_around_the_ways_of_sharing_units(width, batch, Hq, Hkv):
    """The row kernel shares its units out by the table's width; every sequence
    fills its own part of it, one all of it."""
    rng = np.random.default_rng(width)
    full = (width - 1) * 16  # Case gives the table one entry more than the longest needs
    ctx = [max(full - 1, 0)] + rng.integers(0, max(full, 1), batch - 1).tolist()
    new = [1 if full else 0] + [1] * (batch - 1) if full else [1] * batch
    c = Case(ctx, new, Hq, Hkv, 64, "bf16", seed=width)
    assert c.run() == 0
    c.check()
    short = [i for i in range(batch) if ctx[i] < 200][:3]
    if batch > 1 and short:  # and with chunks among them
        new = [40 if i in short else n for i, n in enumerate(new)]
        c = Case(ctx, new, Hq, Hkv, 64, "fp16", seed=width + 1)
        assert c.run() == 0
        c.check()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("Hq,Hkv,new", [(16, 2, 1), (8, 1, 1), (6, 2, 2), (14, 2, 1), (8, 8, 8), (18, 2, 1), (5, 5, 9)])
@pytest.mark.parametrize("longest,batch", [(600, 7), (977, 7), (1900, 2), (1900, 1), (7900, 1)])
def test_units_shared_by_a_block(Hq, Hkv, new, dtype, D, longest, batch):
    """Up to eight rows of a unit: the warps of a block, or of a cluster of 2, 4 or
    8, share it, some of them nothing of the short ones.  (Nine rows: one more than
    they share.)"""
    c = Case([longest, 0, 1, 110, 128, 15, 500][:batch], [new] * batch, Hq, Hkv, D, dtype, seed=Hq + new)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("Hq,Hkv,new", [
    (32, 1, [1, 1, 1, 1]), (20, 1, [1, 1, 1, 1]), (16, 4, [5, 8, 1, 4]), (14, 2, [4, 3, 1, 2]), (3, 1, [10, 6, 5, 0]),
    (8, 2, [8, 200, 1, 9]), (32, 1, [1, 0, 90, 1]), (8, 8, [32, 17, 16, 33]),
])
@pytest.mark.parametrize("ctx,window,sink", [([40, 0, 3, 200], 0, 0), ([1300, 900, 31, 0], 0, 0), ([1300, 900, 31, 700], 100, 7),
                                             ([9000, 33, 2000, 5], 0, 0)])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_up_to_32_rows(Hq, Hkv, new, ctx, window, sink, dtype, D):
    """17 to 32 rows per KV head: two units of 16, with other lengths among them."""
    c = Case(ctx, new, Hq, Hkv, D, dtype, window=window, sink=sink, seed=Hq + sum(new))
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("batch,Hkv,longest", [(60, 4, 1500), (76, 4, 600), (130, 2, 4000), (90, 2, 1500), (610, 4, 520)])
@pytest.mark.parametrize("window,sink", [(0, 0), (200, 20)])
def test_more_units_than_blocks(batch, Hkv, longest, window, sink):
    """In rounds that are nearly full, and in rounds that are not; idle and short
    sequences among them."""
    rng = np.random.default_rng(batch)
    ctx = rng.integers(0, longest, batch)
    ctx[rng.random(batch) < 0.2] = 3
    ctx[batch // 2] = longest
    new = np.where(rng.random(batch) < 0.1, 0, 1)
    new[0] = 1
    c = Case(ctx.tolist(), new.tolist(), Hkv * 4, Hkv, 64, "bf16", window=window, sink=sink, seed=batch)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("new", [[40, 1, 70, 1, 3, 130], [1, 40], [0, 33, 1, 0]])
def test_short_contexts_of_both_kinds(new):
    """Whole units in both kernels: nothing is merged."""
    ctx = [100, 0, 15, 300, 31, 64][:len(new)]
    c = Case(ctx, new, 8, 2, 128, "bf16", seed=21, extra_rows=3)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("ctx,new", [
    ([3000] * 40 + [0], [1] * 40 + [17]),                    # hardly any chunk: most SMs read tokens' pages
    ([600] + [0], [1] + [1500]),                             # hardly a page
    ([0, 2000, 17], [700, 400, 1]), ([5000, 1300], [33, 4]),  # whole units and cut ones
    ([700, 0, 1200], [1, 0, 2]),                             # a chunk announced, none there
    ([700, 40, 1200], [30, 0, 64]),                          # no short ones
    ([100, 900, 0] * 25, [1, 40, 5] * 25),                   # more sequences than a warp looks at in one round
])
@pytest.mark.parametrize("Hq,Hkv,D,window", [(8, 2, 128, 0), (12, 4, 64, 700), (32, 8, 64, 0)])
def test_both_kinds_beside_each_other(ctx, new, Hq, Hkv, D, window):
    c = Case(ctx, new, Hq, Hkv, D, "bf16", window=window, sink=9 if window else 0, seed=sum(new) + Hq)
    assert c.run(max_tokens=max(new) + 20) == 0
    c.check()


@pytest.mark.parametrize("lens", [
    [1024] * 8, [2048], [128] * 33, [700, 0, 20, 1500, 5], [300, 17, 0] * 30, [40] * 100 + [0] * 40 + [600, 90],
])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(32, 8, 64, "fp16"), (12, 3, 128, "bf16")])
def test_more_row_groups_than_blocks(lens, Hq, Hkv, D, dtype):
    """Whole units taken one after another, in any order, with contexts of
    different lengths; twice with the same workspace and the same bits."""
    ctx = [(37 * i) % 500 for i in range(len(lens))]
    c = Case(ctx, lens, Hq, Hkv, D, dtype, seed=len(lens))
    p = c.params()
    outs = []
    for _ in range(3):
        c.out.fill_(7.0)
        sv.sv_chunk_attention(p)
        torch.cuda.synchronize()
        assert sv.sv_get_device_error(c.ws) == 0
        outs.append(c.out.clone())
    c.check()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert not c.ws[:256].any()


@pytest.mark.parametrize("batch,longest", [(3, 10), (3, 900), (50, 900), (400, 100), (3, 9000)])
def test_bad_lengths_and_pages_in_every_way_of_sharing(batch, longest):
    """A sequence with a wrong length is left out, one with a wrong page id reads
    zeros there; the others' results stay."""
    rng = np.random.default_rng(batch + longest)
    ctx = rng.integers(0, longest, batch).tolist()
    ctx[1] = longest
    c = Case(ctx, [1] * batch, 16, 4, 64, "bf16", seed=longest)
    assert c.run() == 0
    want = c.out.clone()
    for at in (0, batch - 1):
        keep = c.lens[at].clone()
        for bad in (100000, -1):
            c.lens[at] = bad
            c.out.fill_(7.0)
            assert c.run() == sv.SV_DEVERR_BAD_LENGTH
            assert (c.out[at] == 7.0).all()
            rest = torch.arange(batch, device="cuda") != at
            # cut units move with the lengths, so both are off by the bound above: 2^-8 (A + |out|) + 2e-4 A
            # each, A at most the largest |v|; 2 x 2e-4 A is less than a tenth of 2^-7 A
            most = torch.nan_to_num(c.v.float()).abs().max()
            diff = (c.out[rest].float() - want[rest].float()).abs()
            assert (diff <= 1.1 * 2.0 ** -7 * (most + want[rest].float().abs())).all()
        c.lens[at] = keep
    page = c.table[1, 0].clone()
    for bad in (c.pages, -7):
        c.table[1, 0] = bad
        assert c.run() == sv.SV_DEVERR_BAD_PAGE
        rest = torch.arange(batch, device="cuda") != 1
        assert torch.equal(c.out[rest], want[rest]) and torch.isfinite(c.out.float()).all()
    c.table[1, 0] = page
    assert c.run() == 0 and torch.equal(c.out, want)


def test_many_sequences():
    rng = np.random.default_rng(5)
    ctx = rng.integers(0, 60, 300).tolist()
    c = Case(ctx, [1] * 300, 4, 2, 64, "bf16", seed=5)
    assert c.run() == 0
    c.check()
    new = rng.integers(0, 40, 300).tolist()
    c = Case(ctx, new, 4, 2, 64, "fp16", seed=6)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("new", [[1], [1, 2], [5, 1], [30]])
def test_rows_behind_the_batch_do_not_count_as_tokens(new):
    """total_tokens (rows of q) may exceed cu_tokens[B]: short sequences are
    still found."""
    c = Case([50, 20][:len(new)], new, 8, 2, 128, "bf16", extra_rows=40, seed=17)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_strided_rows_scale_and_rows_behind_the_batch(new):
    c = Case([50, 20], new, 8, 2, 64, "bf16", q_pad=4, extra_rows=5, seed=7)
    assert c.run(sm_scale=0.3) == 0
    c.check(sm_scale=0.3)
    whole = c.out.as_strided((c.out.shape[0], 12, 64), (12 * 64, 64, 1))
    assert (whole[:, 8:] == 7.0).all()  # the padding between rows


def test_large_scores_and_one_dominant_key():
    for new in ([1], [70]):
        c = Case([300], new, 8, 2, 128, "bf16", seed=8)
        c.q.mul_(20.0)
        assert c.run() == 0
        f = lambda t: t.float().cpu().numpy()  # noqa: E731
        want, lse = oracle.chunk_attention(f(c.q), np.nan_to_num(f(c.k)), np.nan_to_num(f(c.v)), c.table.cpu().numpy(),
                                           c.ctx, c.cu_np)
        # scores up to 20 x 12: their 32-bit sums are off by at most 20 x 1e-4, and a weight's relative error is that
        np.testing.assert_allclose(c.lse.cpu().numpy(), lse, atol=2e-3)
        assert np.abs(f(c.out) - want).max() <= (2 ** -8 + 4e-3) * 2 * np.nan_to_num(np.abs(f(c.v))).max()


def test_results_do_not_depend_on_the_run():
    c = Case([3000, 70, 0], [1, 300, 20], 32, 8, 128, "bf16", seed=9)
    c.run()
    first, first_lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.run()
        assert torch.equal(c.out, first) and torch.equal(c.lse, first_lse)


def test_pages_past_32_bit_offsets():
    pages, Hkv, D = 140000, 8, 128  # 4.6 GB per pool
    k = torch.empty((pages, Hkv, 16, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = Case([70, 33], [1, 90], 16, Hkv, D, "bf16", seed=10, extra_pages=0)
    at = torch.arange(small.pages, device="cuda") + (pages - small.pages)
    k[at], v[at] = small.k, small.v
    assert small.run() == 0
    want, want_lse = small.out.clone(), small.lse.clone()
    small.out.fill_(7.0)
    table = torch.where(small.table >= 0, small.table + (pages - small.pages), -1)
    assert small.run(k_cache=k, v_cache=v, block_table=table) == 0
    assert torch.equal(small.out, want) and torch.equal(small.lse, want_lse)


def test_other_stream_and_captured_graph():
    c = Case([500, 40], [1, 200], 32, 8, 128, "bf16", seed=11)
    assert c.run() == 0
    want = c.out.clone()
    p = c.params()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.out.fill_(0)
        sv.sv_chunk_attention(p)
    s.synchronize()
    assert torch.equal(c.out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.sv_chunk_attention(p)
    # new values in the captured buffers: another table order and other lengths
    other = Case([500, 40], [1, 200], 32, 8, 128, "bf16", seed=12)
    for a, b in ((c.q, other.q), (c.k, other.k), (c.v, other.v), (c.table, other.table)):
        a.copy_(b)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    other.run()
    assert torch.equal(c.out, other.out)
    assert sv.sv_get_device_error(c.ws) == 0


def test_a_call_on_another_current_device_is_refused():
    c = Case([40], [1], 8, 2, 64, "bf16", seed=15)
    p = c.params()

    class Elsewhere:  # q as a tensor of the second GPU would answer
        is_cuda, device = True, "cuda:1"

        def get_device(self):
            return 1

    p.tensors = (Elsewhere(),) + p.tensors[1:]
    with pytest.raises(ValueError, match="cuda:1"):
        sv.sv_chunk_attention(p)


def test_one_workspace_for_calls_of_many_shapes():
    """Nothing in a workspace has to survive from call to call."""
    cases = [Case([900, 3], [1, 1], 8, 2, 64, "bf16", seed=18), Case([900, 3, 200], [70, 1, 1], 32, 8, 128, "fp16", seed=19),
             Case([0], [300], 6, 2, 64, "bf16", seed=20)]
    params = [c.params() for c in cases]
    size = max(c.ws.numel() for c in cases)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    for _ in range(2):
        for c, p in zip(cases, params):
            c.out.fill_(7.0)
            p.workspace, p.workspace_bytes = ws.data_ptr(), size
            sv.sv_chunk_attention(p)
            torch.cuda.synchronize()
            assert sv.sv_get_device_error(ws) == 0
            c.check()


def test_bad_lengths_and_pages_are_reported():
    c = Case([40, 20, 30], [1, 1, 50], 8, 2, 64, "bf16", seed=13)
    assert c.run() == 0
    want = c.out.clone()
    # a context longer than its table, a negative one: those sequences are left out
    for bad in (100000, -1):
        c.lens[0] = bad
        c.out.fill_(7.0)
        assert c.run() == sv.SV_DEVERR_BAD_LENGTH
        assert (c.out[0] == 7.0).all() and torch.equal(c.out[1:], want[1:])
    c.lens[0] = 40
    # more new tokens than max_tokens announced
    # (the others may go to another kernel than with the right number: held to
    # the oracle, not to the first call's bits)
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    assert c.run(max_tokens=20) == sv.SV_DEVERR_BAD_LENGTH
    c.check(rows=2)
    # a page outside the pool reads as zeros; the other sequences are untouched
    for b in (0, 2):
        keep = c.table[b, 0].clone()
        for page in (c.pages, -5, 1 << 30):
            c.table[b, 0] = page
            assert c.run() == sv.SV_DEVERR_BAD_PAGE
            rows = torch.ones(c.T, dtype=torch.bool)
            rows[c.cu_np[b]:c.cu_np[b + 1]] = False
            assert torch.equal(c.out[rows.cuda()], want[rows.cuda()])
            assert torch.isfinite(c.out.float()).all()
        c.table[b, 0] = keep
    assert c.run() == 0 and torch.equal(c.out, want)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("layers,Hkv,D,ctx,new", [
    (1, 2, 64, [0], [1]), (3, 8, 128, [15, 16, 0, 100], [1, 1, 1, 1]), (2, 3, 24, [5, 0, 31], [40, 0, 17]),
    (1, 1, 8, [0] * 70, [1] * 70), (1, 16, 128, [3], [333]), (5, 2, 64, [0, 7], [0, 9]),
])
@pytest.mark.parametrize("fused", [0, 3])
def test_append_matches_the_oracle_bit_for_bit(layers, Hkv, D, ctx, new, fused):
    g = torch.Generator().manual_seed(sum(new))
    need = [-(-(c + n) // 16) for c, n in zip(ctx, new)]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(ctx), max(need) + 1), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    kc, vc = (torch.randint(-32768, 32767, (layers, pages, Hkv, 16, D), generator=g, dtype=torch.int16) for _ in range(2))
    T = sum(new)
    rows = torch.randint(-32768, 32767, (layers, T + 3, fused + 2 * Hkv, D), generator=g, dtype=torch.int16)
    k, v = rows[:, :, fused:fused + Hkv], rows[:, :, fused + Hkv:]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    want = oracle.kv_append(k.numpy(), v.numpy(), kc.numpy(), vc.numpy(), table.numpy(), ctx, cu)
    dev = rows.cuda().view(torch.float16)
    kd, vd = dev[:, :, fused:fused + Hkv], dev[:, :, fused + Hkv:]
    kcd, vcd = kc.cuda().view(torch.float16), vc.cuda().view(torch.float16)
    lens, after = torch.tensor(ctx, dtype=torch.int32).cuda(), torch.zeros(len(ctx), dtype=torch.int32).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.sv_kv_append(kd, vd, kcd, vcd, table.cuda(), lens, torch.from_numpy(cu).cuda(), new_ctx_lens=after, workspace=ws)
    assert sv.sv_get_device_error(ws) == 0
    np.testing.assert_array_equal(kcd.view(torch.int16).cpu().numpy(), want[0])
    np.testing.assert_array_equal(vcd.view(torch.int16).cpu().numpy(), want[1])
    np.testing.assert_array_equal(after.cpu().numpy(), want[2])


def test_append_leaves_out_what_does_not_fit():
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.ones((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    after = torch.zeros(2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([30, 2], dtype=torch.int32, device="cuda")  # 30 + 4 > 2 pages
    sv.sv_kv_append(k, k, kc, vc, table, lens, cu, new_ctx_lens=after, workspace=ws)
    assert sv.sv_get_device_error(ws) == sv.SV_DEVERR_BAD_LENGTH
    assert after.tolist() == [30, 4] and kc[:2].abs().sum() == 0 and kc[2, :, 2:4].eq(1).all()
    assert kc.sum() == 2 * 2 * 64
    lens = torch.tensor([0, 15], dtype=torch.int32, device="cuda")  # slot 16 lies in page 9 of 4
    sv.sv_kv_append(k, k, kc, vc, table, lens, cu, new_ctx_lens=after, workspace=ws)
    assert sv.sv_get_device_error(ws) == sv.SV_DEVERR_BAD_PAGE
    assert kc[2, :, 15].eq(1).all() and kc[0, :, :4].eq(1).all() and kc[3].abs().sum() == 0


def test_append_past_the_last_slot():
    """A table of 2^27 + 1 pages has room for it, a 32-bit slot does not."""
    kc = torch.zeros((4, 1, 16, 8), dtype=torch.bfloat16, device="cuda")
    k = torch.ones((10, 1, 8), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, (1 << 27) + 1), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    after = torch.zeros(1, dtype=torch.int32, device="cuda")
    for length, fits in ((2 ** 31 - 6, False), (2 ** 31 - 11, True)):
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        sv.sv_kv_append(k, k, kc, kc.clone(), table, lens, cu, new_ctx_lens=after, workspace=ws)
        assert sv.sv_get_device_error(ws) == (0 if fits else sv.SV_DEVERR_BAD_LENGTH)
        assert after.item() == (length + 10 if fits else length)
        assert kc.float().sum().item() == (80 if fits else 0)


def test_prompt_then_tokens_then_a_tree():
    """Append and chunk attention fill the cache that tree verification then
    reads: the root's row of the tree equals the next token's."""
    Hq, Hkv, D = 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(14)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    kc, vc = new(8, Hkv, 16, D), new(8, Hkv, 16, D)
    table = torch.tensor([[5, 2, 7, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    after = torch.zeros_like(lens)
    ws = None
    ks, vs, qs, outs = [], [], [], []
    for n in (37, 1, 1):
        k, v, q = new(n, Hkv, D), new(n, Hkv, D), new(n, Hq, D)
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        sv.sv_kv_append(k, v, kc, vc, table, lens, cu, new_ctx_lens=after)
        out = torch.empty_like(q)
        p = sv.make_chunk_params(q=q, k_cache=kc, v_cache=vc, block_table=table, ctx_lens=lens, cu_tokens=cu, out=out,
                                 max_tokens=n)
        ws = torch.zeros(sv.sv_chunk_attention_workspace_size(p), dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = ws.data_ptr(), ws.numel()
        sv.sv_chunk_attention(p)
        assert sv.sv_get_device_error(ws) == 0
        ks.append(k), vs.append(v), qs.append(q), outs.append(out)
        lens.copy_(after)
    # the last token again, as the root of a one-node tree over the 38 tokens before it
    lens.fill_(38)
    out = torch.empty_like(qs[-1])
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    root = torch.tensor([-1], dtype=torch.int32, device="cuda")
    t = sv.make_attn_params(q=qs[-1], tree_k=ks[-1], tree_v=vs[-1], k_cache=kc, v_cache=vc, block_table=table,
                            ctx_lens=lens, cu_nodes=cu, parents=root, out=out, total_nodes=1, max_nodes=1)
    tws = torch.zeros(sv.sv_tree_attention_workspace_size(t), dtype=torch.uint8, device="cuda")
    t.workspace, t.workspace_bytes = tws.data_ptr(), tws.numel()
    sv.sv_tree_attention(t)
    torch.cuda.synchronize()
    # and the whole text at once in float64
    f = lambda x: torch.cat(x).double().cpu()  # noqa: E731
    K, V, Q = f(ks), f(vs), f(qs)
    s = torch.einsum("ihd,jhd->hij", Q, K.repeat_interleave(Hq // Hkv, 1)) / D ** 0.5
    s = s.masked_fill(torch.ones(39, 39, dtype=torch.bool).triu(1), -torch.inf)
    p64 = s.softmax(-1)
    want = torch.einsum("hij,jhd->ihd", p64, V.repeat_interleave(Hq // Hkv, 1))
    mean = torch.einsum("hij,jhd->ihd", p64, V.abs().repeat_interleave(Hq // Hkv, 1))
    tol = 2.0 ** -8 * (mean + want.abs()) * 1.001 + 2e-4 * mean
    worst = ((f(outs) - want).abs() / tol).max().item()
    assert worst <= 1.0
    # the tree kernel merges bf16 partials: one more rounding of the output
    worst = ((out.double().cpu() - want[-1:]).abs() / (tol[-1:] + 2.0 ** -8 * mean[-1:])).max().item()
    assert worst <= 1.0
