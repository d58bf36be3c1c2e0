"""Page bookkeeping and the page copy through the binding, against the pool in
plain Python: every table, count and list equal."""

import random

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_lib()


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class DevicePool:
    def __init__(self, rows, width, pages, page_size=16, Hkv=2, D=16, layers=2):
        self.rows, self.width, self.pages, self.page = rows, width, pages, page_size
        self.model = oracle.Pool([[-1] * width for _ in range(rows)], [0] * rows, [0] * rows, [0] * pages, page_size)
        self.table, self.held = dev(self.model.table), dev(self.model.held)
        self.ctx, self.refs = dev(self.model.ctx), dev(self.model.refs)
        # scratch with whatever another call left in it; only the error word is zero
        self.ws = torch.full((sv.sv_pages_workspace_size(rows, pages),), 0x5A, dtype=torch.uint8, device="cuda")
        self.ws[:256] = 0
        n = max(rows, pages // 2)
        self.src, self.dst = torch.full((n,), -1, dtype=torch.int32, device="cuda"), torch.full((n,), -1, dtype=torch.int32, device="cuda")
        self.count, self.live = dev([0]), dev([0])
        g = torch.Generator(device="cuda").manual_seed(pages)
        shape = (layers, pages, Hkv, page_size, D)
        self.k = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        self.v = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def same(self):
        assert self.table.tolist() == self.model.table
        assert self.held.tolist() == self.model.held
        assert self.ctx.tolist() == self.model.ctx
        assert self.refs.tolist() == self.model.refs

    def error(self):
        return sv.sv_get_device_error(self.ws)

    def reserve(self, new):
        sv.sv_pages_reserve(self.ctx, dev(new), self.table, self.held, self.refs, self.src, self.dst, self.count,
                            page_size=self.page, workspace=self.ws)
        return self.pairs()

    def pairs(self):
        n = int(self.count.item())
        return list(zip(self.src[:n].tolist(), self.dst[:n].tolist()))

    def copy(self, pairs):
        k, v = (oracle.copy_pages(x.view(torch.int16).cpu().numpy(), pairs) for x in (self.k, self.v))
        sv.sv_pages_copy(self.k, self.v, self.src, self.dst, self.count, workspace=self.ws)
        np.testing.assert_array_equal(self.k.view(torch.int16).cpu().numpy(), k)
        np.testing.assert_array_equal(self.v.view(torch.int16).cpu().numpy(), v)

    def set_ctx(self, lens):
        self.model.ctx = list(lens)
        self.ctx.copy_(dev(lens))


@pytest.mark.parametrize("seed,rows,width,pages,page", [(0, 5, 9, 40, 16), (1, 1, 4, 3, 16), (2, 40, 20, 700, 16), (6, 16, 9, 1024, 16),
                                                         (7, 17, 9, 1024, 16), (8, 32, 9, 1024, 16), (9, 33, 9, 1024, 16),
                                                         (3, 7, 33, 97, 1), (4, 300, 40, 5000, 5), (5, 600, 3, 1111, 64)])
def test_random_lives_match_the_pool(seed, rows, width, pages, page):
    rng = random.Random(seed)
    d = DevicePool(rows, width, pages, page)
    m = d.model
    for step in range(25):
        what = rng.choice(["grow", "grow", "fork", "release", "compact"])
        if what == "grow":
            new = [min(c + rng.choice([0, 0, 1, page, 3 * page + 1]), width * page) for c in m.ctx]
            try:
                want = m.reserve(new)
            except MemoryError:
                assert d.reserve(new) == [] and d.error() == sv.SV_DEVERR_NO_PAGES
                d.same()
                continue
            assert d.reserve(new) == want
            d.copy(want)
            d.set_ctx([max(c, n) for c, n in zip(m.ctx, new)])
        elif what == "fork":
            empty = [b for b in range(rows) if m.held[b] == 0]
            rng.shuffle(empty)
            children = empty[:rng.randrange(0, len(empty) + 1)]
            others = [b for b in range(rows) if b not in children]
            if not others or not children:
                continue
            parents = [rng.choice(others) for _ in children]
            m.fork(parents, children)
            sv.sv_pages_fork(dev(parents), dev(children), d.table, d.ctx, d.held, d.refs, page_size=page, workspace=d.ws)
        elif what == "release":
            keep = [rng.choice([c, c, c // 2, 0]) for c in m.ctx]
            m.release(keep)
            sv.sv_pages_release(dev(keep), d.table, d.held, d.refs, page_size=page, workspace=d.ws)
            d.set_ctx(keep)
        else:
            before = d.table.clone(), d.refs.clone()
            apart = rng.random() < 0.5
            table, refs = (torch.full_like(d.table, 99), torch.full_like(d.refs, 99)) if apart else (d.table, d.refs)
            want, live = m.compact()
            sv.sv_pages_compact(d.table, d.held, d.refs, table, refs, d.src, d.dst, d.count, d.live, workspace=d.ws)
            assert d.pairs() == want and int(d.live.item()) == live
            if apart:
                assert torch.equal(d.table, before[0]) and torch.equal(d.refs, before[1])
                d.table, d.refs = table, refs
            d.copy(want)
        assert d.error() == 0
        d.same()
        m.check()


@pytest.mark.parametrize("pages", [31, 32, 33, 255, 256, 257, 1024, 1025, 8193, 2097152])
def test_pool_sizes_around_the_bitmap_words(pages):
    """The last pages of the pool are found and moved."""
    d = DevicePool(2, 40, pages, Hkv=1, D=8, layers=1) if pages < 10000 else None
    if d is None:  # bookkeeping only, no caches
        d = DevicePool(2, 40, 33, Hkv=1, D=8, layers=1)
        d.pages = pages
        d.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        d.src = torch.full((pages // 2,), -1, dtype=torch.int32, device="cuda")
        d.dst = d.src.clone()
        d.ws = torch.zeros(sv.sv_pages_workspace_size(2, pages), dtype=torch.uint8, device="cuda")
    d.refs.fill_(1)
    d.refs[-3:] = 0
    assert d.reserve([33, 0]) == [] and d.error() == 0
    assert d.table[0, :4].tolist() == [pages - 3, pages - 2, pages - 1, -1] and d.refs[-3:].tolist() == [1, 1, 1]
    assert d.reserve([0, 1]) == [] and d.error() == sv.SV_DEVERR_NO_PAGES
    d.refs[:-2] = 0  # only the last two stay: they move to the front
    d.held.copy_(dev([3, 0]))
    d.table[0, 0] = pages - 1
    d.refs[-1] = 2
    sv.sv_pages_compact(d.table, d.held, d.refs, d.table, d.refs, d.src, d.dst, d.count, d.live, workspace=d.ws)
    assert d.pairs() == [(pages - 2, 0), (pages - 1, 1)] and int(d.live.item()) == 2 and d.error() == 0
    assert d.table[0, :3].tolist() == [1, 0, 1] and d.refs[:3].tolist() == [1, 2, 0] and int(d.refs.sum()) == 3


def test_bad_state_is_reported_and_left_alone():
    d = DevicePool(4, 6, 32)
    d.reserve([40, 20, 0, 0])
    d.model.reserve([40, 20, 0, 0])
    d.set_ctx([40, 20, 0, 0])
    d.same()
    call = lambda p, c: sv.sv_pages_fork(dev(p), dev(c), d.table, d.ctx, d.held, d.refs, workspace=d.ws)  # noqa: E731
    for parents, children in (([0], [0]), ([0], [9]), ([-1], [2]), ([0], [1])):  # itself, outside, a child with pages
        call(parents, children)
        assert d.error() == sv.SV_DEVERR_BAD_ROW
        d.same()
    call([0, 1], [2, 2])  # one child twice: the first pair has it
    assert d.error() == sv.SV_DEVERR_BAD_ROW
    d.model.fork([0], [2])
    d.same()
    call([2, 1], [3, 2])  # the parent is another pair's child (and that child holds pages)
    assert d.error() == sv.SV_DEVERR_BAD_ROW
    d.same()
    # longer than the table: that row alone takes no part
    assert d.reserve([41, 6 * 16 + 1, 0, 0]) == [(2, 5)] and d.error() == sv.SV_DEVERR_BAD_LENGTH
    assert d.model.reserve([41, 0, 0, 0]) == [(2, 5)]
    d.same()
    # a held entry that names no page
    d.table[1, 1] = -1
    d.ctx[1] = 20
    before = d.table.clone()
    assert d.reserve([0, 30, 0, 0]) == [] and d.error() == sv.SV_DEVERR_BAD_PAGE
    assert torch.equal(d.table, before)
    sv.sv_pages_compact(d.table, d.held, d.refs, d.table, d.refs, d.src, d.dst, d.count, d.live, workspace=d.ws)
    assert d.error() == sv.SV_DEVERR_BAD_PAGE
    sv.sv_pages_release(dev([40, 0, 40, 0]), d.table, d.held, d.refs, workspace=d.ws)
    assert d.error() == sv.SV_DEVERR_BAD_PAGE and d.held[1].item() == 0 and int(d.refs.min()) == 0
    sv.sv_pages_release(dev([-1, 0, 40, 0]), d.table, d.held, d.refs, workspace=d.ws)
    assert d.error() == sv.SV_DEVERR_BAD_LENGTH
    # copies: a page outside the pool is skipped
    d.src[:2], d.dst[:2] = dev([0, 40]), dev([31, 1])
    d.count.fill_(2)
    k = d.k.clone()
    sv.sv_pages_copy(d.k, d.v, d.src, d.dst, d.count, workspace=d.ws)
    assert d.error() == sv.SV_DEVERR_BAD_PAGE
    k[:, 31] = k[:, 0]
    assert torch.equal(d.k, k)


@pytest.mark.parametrize("shape", [(1, 5, 1, 1, 8), (3, 40, 8, 16, 128), (2, 9, 3, 5, 40), (4, 12, 1, 16, 8)])
def test_copy_of_odd_pages_one_pool_and_a_short_list(shape):
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(shape, generator=g, device="cuda").to(torch.float16)
    want = k.clone()
    src, dst, count = dev([0, 2, 4]), dev([1, 3, 0]), dev([9])  # the list holds three
    for a, z in ((0, 1), (2, 3)):
        want[:, z] = k[:, a]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.sv_pages_copy(k, None, src[:2].contiguous(), dst[:2].contiguous(), count, workspace=ws)
    assert torch.equal(k, want) and sv.sv_get_device_error(ws) == 0
    count.fill_(-4)
    sv.sv_pages_copy(k, None, src, dst, count)
    assert torch.equal(k, want)
    # page summaries [pages, Hkv, 2, D] are a pool of one layer
    s = k[0].contiguous()
    want = s.clone()
    want[3] = s[1]
    sv.sv_pages_copy(s, None, dev([1]), dev([3]), dev([1]))
    assert torch.equal(s, want)


def test_captured_step_replays_on_new_lengths():
    d = DevicePool(3, 8, 40)
    new = dev([20, 33, 0])
    step = lambda: sv.sv_pages_reserve(d.ctx, new, d.table, d.held, d.refs, d.src, d.dst, d.count, workspace=d.ws)  # noqa: E731
    step()
    assert d.model.reserve([20, 33, 0]) == []
    d.set_ctx([20, 33, 0])
    sv.sv_pages_fork(dev([1]), dev([2]), d.table, d.ctx, d.held, d.refs, workspace=d.ws)
    d.model.fork([1], [2])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
        sv.sv_pages_copy(d.k, d.v, d.src, d.dst, d.count, workspace=d.ws)
    d.same()
    for lens in ([25, 35, 40], [50, 35, 90]):
        new.copy_(dev(lens))
        k = d.k.clone()
        g.replay()
        want = d.model.reserve(lens)
        assert d.pairs() == want and d.error() == 0
        for a, z in want:
            assert torch.equal(d.k[:, z], k[:, a])
        d.same()
        d.set_ctx([max(a, b) for a, b in zip(d.model.ctx, lens)])


def test_fork_grow_and_read_through_attention():
    """Two samples of one prompt: forked, grown by different tokens, attended;
    then compacted, and the answers stay."""
    Hq, Hkv, D = 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    d = DevicePool(3, 4, 24, Hkv=Hkv, D=D, layers=1)
    d.k, d.v = new(1, 24, Hkv, 16, D), new(1, 24, Hkv, 16, D)

    def append(k, v, cu, after):
        sv.sv_kv_append(k, v, d.k[0], d.v[0], d.table, d.ctx, dev(cu), new_ctx_lens=after)

    after = torch.zeros_like(d.ctx)
    d.reserve([25, 0, 0])
    k, v = new(25, Hkv, D), new(25, Hkv, D)
    append(k, v, [0, 25, 25, 25], after)
    d.ctx.copy_(after)
    sv.sv_pages_fork(dev([0, 0]), dev([1, 2]), d.table, d.ctx, d.held, d.refs, workspace=d.ws)
    pairs = d.reserve([26, 26, 26])
    assert pairs == [(1, 2), (1, 3)]
    sv.sv_pages_copy(d.k, d.v, d.src, d.dst, d.count, workspace=d.ws)
    k1, v1, q = new(3, Hkv, D), new(3, Hkv, D), new(3, Hq, D)
    append(k1, v1, [0, 1, 2, 3], after)
    assert after.tolist() == [26, 26, 26]

    def attend():
        out = torch.empty_like(q)
        p = sv.make_chunk_params(q=q, k_cache=d.k[0], v_cache=d.v[0], block_table=d.table, ctx_lens=d.ctx,
                                 cu_tokens=dev([0, 1, 2, 3]), out=out, max_tokens=1)
        ws = torch.zeros(sv.sv_chunk_attention_workspace_size(p), dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = ws.data_ptr(), ws.numel()
        sv.sv_chunk_attention(p)
        torch.cuda.synchronize()
        assert sv.sv_get_device_error(ws) == 0
        return out

    out = attend()
    for b in range(3):
        K = torch.cat([k, k1[b:b + 1]]).double().repeat_interleave(Hq // Hkv, 1)
        V = torch.cat([v, v1[b:b + 1]]).double().repeat_interleave(Hq // Hkv, 1)
        w = (torch.einsum("hd,jhd->hj", q[b].double(), K) / D ** 0.5).softmax(-1)
        want, mean = torch.einsum("hj,jhd->hd", w, V), torch.einsum("hj,jhd->hd", w, V.abs())
        assert ((out[b].double() - want).abs() <= 2.0 ** -8 * 1.001 * (mean + want.abs()) + 2e-4 * mean).all()
    sv.sv_pages_release(dev([0, 26, 26]), d.table, d.held, d.refs, workspace=d.ws)
    sv.sv_pages_compact(d.table, d.held, d.refs, d.table, d.refs, d.src, d.dst, d.count, d.live, workspace=d.ws)
    # rows 1 and 2 share page 0 and own 2 and 3: three pages, page 3 moves into the hole at 1
    assert d.live.item() == 3 and d.pairs() == [(3, 1)]
    sv.sv_pages_copy(d.k, d.v, d.src, d.dst, d.count, workspace=d.ws)
    d.table[0, :2] = d.table[1, :2]  # row 0 is attended too: any valid pages
    assert torch.equal(attend()[1:], out[1:]) and d.error() == 0
