"""Tree attention with SV_ATTN_EARLY_CONTEXT right behind the calls that write its
context: append, reserve, fork, compact and the page copy.  With the flag
it reads tables, lengths and pages as soon as it may start, so its result has the
bits of the call without the flag."""

import pytest
import torch

from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib

pytestmark = pytest.mark.gpu

HQ, HKV, D, B, TOKENS = 8, 2, 128, 3, 4000
WIDTH = TOKENS // 16 + 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """A cache of B sequences, a call that writes part of it, and one-node trees
    over it, both in one captured graph."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(5)
        new = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.pages = B * WIDTH + 40
        self.k, self.v = new(self.pages, HKV, 16, D), new(self.pages, HKV, 16, D)
        self.rows = new(2, B * TOKENS, HKV, D)
        self.table = torch.arange(B * WIDTH, dtype=torch.int32, device="cuda").flip(0).view(B, WIDTH).contiguous()
        self.lens, self.held = ints([TOKENS] * B), ints([WIDTH] * B)
        self.refs = torch.zeros(self.pages, dtype=torch.int32, device="cuda")
        self.refs[:B * WIDTH] = 1
        self.src, self.dst = (torch.zeros(self.pages, dtype=torch.int32, device="cuda") for _ in range(2))
        self.count, self.live = ints([0]), ints([0])
        self.ws = torch.zeros(sv.sv_pages_workspace_size(B, self.pages), dtype=torch.uint8, device="cuda")
        self.q, self.tree = new(B, HQ, D), new(2, B, HKV, D)
        self.out = torch.zeros_like(self.q)
        self.cu, self.root = ints(list(range(B + 1))), ints([-1] * B)
        self.state = ("k", "v", "table", "lens", "held", "refs", "src", "dst", "count")

    def attend(self, flags):
        p = sv.make_attn_params(q=self.q, tree_k=self.tree[0], tree_v=self.tree[1], k_cache=self.k, v_cache=self.v,
                                block_table=self.table, ctx_lens=self.lens, cu_nodes=self.cu,
                                parents=self.root, out=self.out, total_nodes=B, max_nodes=1, flags=flags)
        if not hasattr(self, "tws"):
            self.tws = torch.zeros(sv.sv_tree_attention_workspace_size(p), dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = self.tws.data_ptr(), self.tws.numel()
        return p

    def run(self, write):
        before = {n: getattr(self, n).clone() for n in self.state}

        def reset():
            for n, t in before.items():
                getattr(self, n).copy_(t)
            self.out.zero_()

        plain = self.attend(sv.SV_ATTN_KERNEL_PAIRED)
        early = self.attend(sv.SV_ATTN_KERNEL_PAIRED | sv.SV_ATTN_EARLY_CONTEXT)
        write()
        torch.cuda.synchronize()
        sv.sv_tree_attention(plain)
        torch.cuda.synchronize()
        want = self.out.clone()
        assert torch.isfinite(want.float()).all()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            write()
            sv.sv_tree_attention(early)
        for _ in range(20):
            reset()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(self.out, want)
        assert sv.sv_get_device_error(self.ws) == 0 and sv.sv_get_device_error(self.tws) == 0


def test_append():
    s = Step()
    start, cu = ints([0] * B), ints([TOKENS * i for i in range(B + 1)])
    s.lens.zero_()
    s.run(lambda: sv.sv_kv_append(s.rows[0], s.rows[1], s.k, s.v, s.table, start, cu, new_ctx_lens=s.lens, workspace=s.ws))


def test_reserve():
    s = Step()
    empty = ints([0] * B)
    s.table.fill_(-1)
    s.held.zero_()
    s.refs.zero_()
    s.run(lambda: sv.sv_pages_reserve(empty, s.lens, s.table, s.held, s.refs, s.src, s.dst, s.count, workspace=s.ws))


def test_fork():
    s = Step()
    parents, children = ints([0, 0]), ints([1, 2])
    s.table[1:] = -1
    s.held[1:] = 0
    s.lens[1:] = 0
    s.refs.zero_()
    s.refs[s.table[0].long()] = 1
    s.run(lambda: sv.sv_pages_fork(parents, children, s.table, s.lens, s.held, s.refs, workspace=s.ws))


def test_compact():
    s = Step()
    s.table.add_(40)
    s.refs.zero_()
    s.refs[40:] = 1

    def write():  # the table after the moves, then the moves
        sv.sv_pages_compact(s.table, s.held, s.refs, s.table, s.refs, s.src, s.dst, s.count, s.live, workspace=s.ws)
        sv.sv_pages_copy(s.k, s.v, s.src, s.dst, s.count, workspace=s.ws)

    s.run(write)
