"""Attention over shared prefixes through the binding, against the float64 oracle
of chunk attention (what is shared does not show in the result).

Tolerances as derived for chunk attention: each weight is rounded to the 16-bit
type once (half a step, eps / 2, relative) and the output once; scores, sums and
partial rows are 32-bit (1e-4 of lse, 2e-4 of the mean of |v|)."""

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
    """groups: lists of (own context behind the prefix, new tokens); prefixes: shared tokens, whole pages.  Slots no row
    may read hold NaN; entries of shared pages name them in a group's first row alone, -1 in the others."""

    def __init__(self, prefixes, groups, Hq, Hkv, D, dtype="bf16", seed=0, q_pad=0, extra_rows=0, all_rows=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.Hq, self.Hkv, self.D = DTYPES[dtype], Hq, Hkv, D
        seqs = [(p, own, new) for p, members in zip(prefixes, groups) for own, new in members]
        self.ctx = [p + own for p, own, _ in seqs]
        self.new = [new for _, _, new in seqs]
        self.B, self.T = len(seqs), sum(self.new)
        need = [-(-(c + n) // 16) for c, n in zip(self.ctx, self.new)]
        self.pages = sum(p // 16 for p in prefixes) + sum(k - p // 16 for k, (p, _, _) in zip(need, seqs)) + 3
        order = iter(rng.permutation(self.pages).tolist())
        width = max(max(need), max(prefixes) // 16, 1) + 1
        table = np.full((self.B, width), -1, dtype=np.int32)
        k = torch.full((self.pages, Hkv, 16, D), float("nan"))
        v = torch.full((self.pages, Hkv, 16, D), float("nan"))

        def fill(page, rows):
            k[page, :, :rows] = torch.randn((Hkv, rows, D), generator=g)
            v[page, :, :rows] = torch.randn((Hkv, rows, D), generator=g)

        b = 0
        for p, members in zip(prefixes, groups):
            shared = [next(order) for _ in range(p // 16)] if members else []
            for page in shared:
                fill(page, 16)
            for _ in members:
                table[b, :p // 16] = shared
                for lp in range(p // 16, need[b]):
                    table[b, lp] = next(order)
                    fill(table[b, lp], min(16, self.ctx[b] + self.new[b] - lp * 16))
                b += 1
        self.table_np = table
        rows = self.T + extra_rows
        wide = torch.randn((rows, Hq + q_pad, D), generator=g).to(self.dtype).cuda()
        self.q = wide[:, :Hq]
        self.k, self.v = k.to(self.dtype).cuda(), v.to(self.dtype).cuda()
        self.table = torch.from_numpy(table).cuda()
        self.cu_np = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.cu = torch.from_numpy(self.cu_np).cuda()
        self.lens = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.cu_groups = torch.tensor(np.concatenate([[0], np.cumsum([len(m) for m in groups])]), dtype=torch.int32).cuda()
        self.prefix = torch.tensor(prefixes, dtype=torch.int32, device="cuda")
        self.most = max(self.new)
        self.most_of_group = max(sum(n for _, n in m) for m in groups)
        self.out = torch.full((rows, Hq + q_pad, D), 7.0, dtype=self.dtype, device="cuda")[:, :Hq]
        self.lse = torch.full((rows, Hq), 7.0, device="cuda")

    def params(self, **kw):
        kw = {**dict(q=self.q, k_cache=self.k, v_cache=self.v, block_table=self.table, ctx_lens=self.lens,
                     cu_tokens=self.cu, cu_groups=self.cu_groups, prefix_lens=self.prefix, out=self.out, lse=self.lse,
                     max_tokens=self.most, max_group_tokens=self.most_of_group), **kw}
        p = sv.make_prefix_params(**kw)
        self.ws = torch.zeros(sv.sv_prefix_attention_workspace_size(p), dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = self.ws.data_ptr(), self.ws.numel()
        return p

    def run(self, **kw):
        sv.sv_prefix_attention(self.params(**kw))
        torch.cuda.synchronize()
        return sv.sv_get_device_error(self.ws)

    def check(self, sm_scale=None, untouched=()):
        f = lambda t: t.float().cpu().numpy()  # noqa: E731
        q, k, v = f(self.q), np.nan_to_num(f(self.k)), np.nan_to_num(f(self.v))
        want, lse = oracle.chunk_attention(q, k, v, self.table_np, self.ctx, self.cu_np, sm_scale=sm_scale)
        mean, _ = oracle.chunk_attention(q, k, np.abs(v), self.table_np, self.ctx, self.cu_np, sm_scale=sm_scale)
        got, got_lse = f(self.out), self.lse.cpu().numpy()
        own = np.zeros(len(got), dtype=bool)
        own[:self.T] = True
        for b in untouched:
            own[self.cu_np[b]:self.cu_np[b + 1]] = False
        half = torch.finfo(self.dtype).eps / 2
        tol = half * (mean + np.abs(want)) * 1.001 + 2e-4 * mean + torch.finfo(self.dtype).tiny
        if own.any():
            worst = (np.abs(got[own] - want[own]) / tol[own]).max()
            assert worst <= 1.0, worst
            assert np.isfinite(got_lse[own]).all() and np.abs(got_lse[own] - lse[own]).max() <= 1e-4
        assert (got[~own] == 7.0).all() and (got_lse[~own] == 7.0).all()


HEADS = [(8, 2, 64), (32, 8, 128), (4, 4, 128), (7, 1, 128), (20, 1, 64), (128, 1, 128)]
GROUPS = [
    ([32], [[(5, 1), (0, 1)]]),                                             # two samples, one of them at the prefix's end
    ([16], [[(0, 1)] * 3]),
    ([512], [[(i, 1) for i in range(11)]]),
    ([400, 0, 1008, 48], [[(3, 1), (20, 1)], [(50, 1), (0, 1), (7, 1)], [(i * 9, 1) for i in range(40)], [(33, 1)]]),
    ([160, 320], [[(3, 2), (0, 5), (40, 1)], [(100, 3), (17, 0), (2, 9)]]),  # several new tokens, one sequence with none
    ([640], [[(0, 1), (13, 140), (5, 2), (9, 33)]]),                        # a chunk among single tokens
    ([256, 128], [[(3, 150), (0, 170)], [(1, 1), (2, 1)]]),                 # a group whose chunks are too long to share
    ([128, 96, 64], [[(0, 1), (1, 1)], [], [(4, 1), (60, 2)]]),             # an empty group
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("prefixes,groups", GROUPS)
def test_groups(prefixes, groups, Hq, Hkv, D, dtype):
    c = Case(prefixes, groups, Hq, Hkv, D, dtype, seed=Hq + len(groups))
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("samples", [2, 4, 5, 16, 17, 70])
@pytest.mark.parametrize("prefix", [1024, 5008, 20000])
def test_long_prefixes_are_cut_between_workers(prefix, samples, dtype, D):
    c = Case([prefix], [[(i % 40, 1) for i in range(samples)]], 8, 2, D, dtype, seed=samples)
    assert c.run() == 0
    c.check()


def test_long_tails_of_every_kind():
    c = Case([3008, 1600], [[(2000, 1), (30, 20), (4001, 1), (0, 1)], [(900, 3), (3000, 40)]], 16, 2, 128, "bf16", seed=5)
    assert c.run() == 0
    c.check()


def test_padding_strides_and_scale():
    """Token rows behind the last sequence, many enough that parts go by the sequences' order; q and out are slices."""
    for extra in (3, 900):
        c = Case([160, 64], [[(3, 2), (0, 5), (40, 1)], [(100, 3), (17, 0)]], 8, 2, 64, "bf16", seed=9, q_pad=4, extra_rows=extra)
        assert c.run(sm_scale=0.3) == 0
        c.check(sm_scale=0.3)


def test_without_lse_and_larger_host_bounds():
    c = Case([320], [[(i, 1) for i in range(6)]], 8, 2, 64, seed=2)
    assert c.run(lse=None, max_tokens=50, max_group_tokens=1000) == 0
    out = c.out.clone()
    assert c.run() == 0
    c.check()
    c.out.copy_(out)
    c.check()


def test_groups_of_very_different_sizes():
    """One group of several M tiles among many small ones, its bound and a far larger one."""
    for most in (50, 66, 1 << 20):
        c = Case([64] * 9, [[(i, 1) for i in range(50)]] + [[(3, 1), (20, 1)]] * 8, 32, 8, 128, seed=12)
        assert c.run(max_group_tokens=most) == 0
        c.check()


def test_equals_chunk_attention():
    """Each of the two is off by eps / 2 (A + |out|) + 2e-4 A at most, A the mean of |v| under the weights (itself
    computed to 1 %), so they differ by twice that."""
    c = Case([2000], [[(i * 3, 1) for i in range(24)]], 32, 8, 128, "bf16", seed=4)

    def chunk(v):
        out, lse = torch.empty_like(c.q), torch.empty_like(c.lse)
        p = sv.make_chunk_params(q=c.q, k_cache=c.k, v_cache=v, block_table=c.table, ctx_lens=c.lens, cu_tokens=c.cu,
                                 out=out, lse=lse, max_tokens=1)
        ws = torch.zeros(sv.sv_chunk_attention_workspace_size(p), dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = ws.data_ptr(), ws.numel()
        sv.sv_chunk_attention(p)
        return out.float(), lse

    assert c.run() == 0
    ref, lse = chunk(c.v)
    mean = 1.01 * chunk(c.v.abs())[0]
    assert (c.lse - lse).abs().max() <= 2e-4
    assert ((c.out.float() - ref).abs() <= 2 * (2.0 ** -8 * 1.001 * (mean + ref.abs()) + 2e-4 * mean)).all()


def test_same_bits_on_every_run_and_workspace():
    c = Case([4000, 480], [[(i * 7, 1) for i in range(40)], [(5, 3), (90, 1)]], 32, 8, 128, "fp16", seed=6)
    p = c.params()
    sv.sv_prefix_attention(p)
    first, lse = c.out.clone(), c.lse.clone()
    for _ in range(4):
        c.out.fill_(7.0)
        sv.sv_prefix_attention(p)
        assert torch.equal(first, c.out) and torch.equal(lse, c.lse)
    # the same workspace for another call in between
    d = Case([64], [[(1, 1), (30, 2)]], 32, 8, 128, "fp16", seed=7)
    small = d.params()
    assert c.ws.numel() >= d.ws.numel()
    small.workspace, small.workspace_bytes = c.ws.data_ptr(), c.ws.numel()
    sv.sv_prefix_attention(small)
    torch.cuda.synchronize()
    d.check()
    c.out.fill_(7.0)
    sv.sv_prefix_attention(p)
    assert torch.equal(first, c.out) and sv.sv_get_device_error(c.ws) == 0


def test_lengths_that_do_not_fit():
    groups = ([160, 64], [[(3, 1), (0, 1), (40, 1)], [(100, 1), (17, 1)]])
    c = Case(*groups, 8, 2, 64, seed=3)
    c.lens[1] = 150  # shorter than its group's prefix
    assert c.run() == sv.SV_DEVERR_BAD_LENGTH
    c.check(untouched=[1])
    for bad, out in (((0, 161), [0, 1, 2]), ((0, -16), [0, 1, 2]), ((1, 1 << 20), [3, 4])):  # a prefix of no whole pages, ...
        c = Case(*groups, 8, 2, 64, seed=3)
        c.prefix[bad[0]] = bad[1]
        assert c.run() == sv.SV_DEVERR_BAD_LENGTH
        c.check(untouched=out)
    for cu_groups in ([0, 3, 6], [1, 3, 5], [0, 3, 4], [0, 7, 5], [-1, 3, 5]):  # groups that are not the sequences
        c = Case(*groups, 8, 2, 64, seed=3)
        c.cu_groups.copy_(torch.tensor(cu_groups, dtype=torch.int32))
        assert c.run() == sv.SV_DEVERR_BAD_LENGTH
    c = Case(*groups, 8, 2, 64, seed=3)
    assert c.run(max_group_tokens=2) == sv.SV_DEVERR_BAD_LENGTH  # fewer than the first group has
    c.check(untouched=[0, 1, 2])
    c = Case(*groups, 8, 2, 64, seed=3)
    c.cu[3] = 99
    assert c.run() == sv.SV_DEVERR_BAD_LENGTH


def test_bad_pages_are_reported():
    for samples in (2, 20):
        c = Case([160], [[(3, 1)] * samples], 8, 2, 64, seed=3)
        c.table[0, 4] = c.pages
        assert c.run() == sv.SV_DEVERR_BAD_PAGE
        assert torch.isfinite(c.out.float()).all()


def test_nothing_to_do():
    c = Case([160], [[(3, 1), (4, 1)]], 8, 2, 64, seed=3)
    none = torch.zeros((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    assert c.run(q=none, out=none, lse=None, cu_tokens=torch.zeros_like(c.cu)) == 0
    c.cu.zero_()
    assert c.run() == 0  # every sequence brings nothing
    assert c.out.eq(7).all()


def test_captured_replayed_and_two_streams():
    c = Case([1600], [[(i, 1) for i in range(30)]], 32, 8, 128, "bf16", seed=8)
    p = c.params()
    sv.sv_prefix_attention(p)
    first = c.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_prefix_attention(p)
    c.out.fill_(7.0)
    graph.replay()
    assert torch.equal(first, c.out)
    # two calls at once, each with its own workspace
    d = Case([800], [[(i, 1) for i in range(9)]], 32, 8, 128, "bf16", seed=9)
    pd = d.params()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, x in zip(streams, (p, pd)):
            sv.sv_prefix_attention(x, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)
    d.check()


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 128), (8, 2, 64), (16, 2, 128), (32, 2, 64), (20, 1, 64)])
@pytest.mark.parametrize("each", [1, 2, 4])
def test_padded_decode_steps(each, Hq, Hkv, D):
    """One token per sequence and token rows behind them, as of a step captured for more sequences; the workspace held
    other calls' rows (here NaN, and indices of -1) behind its header."""
    for extra in (0, 1, 2, 4, 12, 40):
        c = Case([48, 0, 1600], [[(5 * i + 1, 1) for i in range(each)]] * 3, Hq, Hkv, D, seed=each + extra, extra_rows=extra)
        p = c.params()
        c.ws[256:] = 255
        sv.sv_prefix_attention(p)
        torch.cuda.synchronize()
        assert sv.sv_get_device_error(c.ws) == 0
        c.check()
    c = Case([320], [[(3, 1), (0, 0), (9, 1)]], Hq, Hkv, D, seed=each, extra_rows=70)  # and one that brings nothing
    p = c.params()
    c.ws[256:] = 255
    sv.sv_prefix_attention(p)
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (32, 8, 128), (16, 1, 128)])
@pytest.mark.parametrize("groups", [[[(3, 1), (0, 1), (9, 1)]] * 3, [[(3, 150), (0, 170)], [(1, 1)], [(4, 70), (60, 1), (2, 2), (9, 300)]]])
def test_shared_pages_are_named_by_the_first_row_alone(groups, Hq, Hkv, D):
    """The entries of a group's other rows for them are not read, whether or not it is worth sharing: here they name no page,
    or another one."""
    for other in (-1, 1 << 30, 0):
        c = Case([160, 64, 1600], groups, Hq, Hkv, D, seed=Hq)
        ends = c.cu_groups.tolist()
        for first, end, prefix in zip(ends, ends[1:], (160, 64, 1600)):
            c.table[first + 1:end, :prefix // 16] = other
        assert c.run() == 0
        c.check()


def test_calls_one_behind_the_other_on_one_workspace():
    """Calls whose work is shared out differently, nothing between them: each sees its own entries and split."""
    cases = [Case([1600, 320], [[(i, 1) for i in range(each)], [(900, 3), (i0, 40)]], 32, 8, 128, seed=each)
             for each, i0 in ((40, 7), (9, 1500), (64, 30))]
    params = [c.params() for c in cases]
    ws = max((c.ws for c in cases), key=lambda t: t.numel())
    first = []
    for c, p in zip(cases, params):
        p.workspace, p.workspace_bytes = ws.data_ptr(), ws.numel()
        sv.sv_prefix_attention(p)
        torch.cuda.synchronize()
        c.check()
        first.append((c.out.clone(), c.lse.clone()))
    for i in range(30):
        for c, p in zip(cases, params):
            sv.sv_prefix_attention(p)
    torch.cuda.synchronize()
    for c, (out, lse) in zip(cases, first):
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    assert sv.sv_get_device_error(ws) == 0


@pytest.mark.parametrize("B,Hq,Hkv", [(1023, 4, 2), (1024, 4, 2), (1025, 4, 1), (2500, 2, 2), (9000, 1, 1)])
def test_more_sequences_than_the_entries_are_made_of_at_once(B, Hq, Hkv):
    """Groups of one to seven sequences (and empty ones), more of them than a block has threads and than fit its staged
    arrays; tokens of every kind among them."""
    rng = np.random.default_rng(B)
    groups, prefixes, left = [], [], B
    while left > 0:
        n = min(left, int(rng.integers(0, 8)))
        if n == 0 and len(groups) % 9:
            continue
        groups.append([(int(rng.integers(0, 40)), int(rng.choice([0, 1, 1, 1, 1, 2, 30]))) for _ in range(n)])
        prefixes.append(16 * int(rng.integers(0, 4)))
        left -= n
    c = Case(prefixes, groups, Hq, Hkv, 64, seed=B, extra_rows=int(rng.integers(0, 100)))
    p = c.params(max_group_tokens=c.most_of_group + 5)
    c.ws[256:] = 255
    sv.sv_prefix_attention(p)
    torch.cuda.synchronize()
    assert sv.sv_get_device_error(c.ws) == 0
    c.check()


def test_cache_offsets_past_32_bits():
    """The pages at the end of a pool of 2.3e9 elements."""
    c = Case([160, 1600], [[(3, 1), (20, 2)], [(i, 1) for i in range(20)] + [(5, 40)]], 32, 8, 128, seed=14)
    first = 140000 - c.pages
    big = [torch.zeros((140000, 8, 16, 128), dtype=c.dtype, device="cuda") for _ in range(2)]
    big[0][first:], big[1][first:] = c.k, c.v
    c.table += first
    assert c.run(k_cache=big[0], v_cache=big[1]) == 0
    c.check()
