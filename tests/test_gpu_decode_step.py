"""The decode step of samples that share a prompt, as a program runs it: prompts
appended and forked, then per step pages reserved and copied, per layer the append
with the rotation and the attention over the shared prefix, and the next tokens
sampled from the logits; eagerly against float64, and captured and replayed.

The cache is compared with a dense float64 history per sequence (keys rotated in
float64, rounded once: half a step, and 5e-7 of the two elements of a pair for the
angle and the products), attention with the oracle on the cache's own values
(tolerance as in the tests of the attention), tokens and shares with the sampling
oracle on the logits that were sampled."""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib

pytestmark = pytest.mark.gpu

LAYERS, HQ, HKV, D, R, V = 2, 8, 2, 64, 32, 500
PROMPTS = [37, 64]                 # a shared page that ends inside, and one that is full
ROWS = [[0, 1, 2], [3, 4, 5, 6, 7]]  # of the table: the prompt's and its samples'
STEPS = 20                         # past the end of a page
SCALE = 0.7


@pytest.fixture(scope="module", autouse=True)
def lib():
    ensure_lib()


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Engine:
    def __init__(self, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = dtype
        self.normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
        self.B = sum(len(r) for r in ROWS)
        pages, width = 40, 8
        self.table = torch.full((self.B, width), -1, dtype=torch.int32, device="cuda")
        self.held, self.ctx, self.after = (torch.zeros(self.B, dtype=torch.int32, device="cuda") for _ in range(3))
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.src, self.dst, self.count = dev([0] * pages), dev([0] * pages), dev([0])
        self.kc = torch.zeros((LAYERS, pages, HKV, 16, D), dtype=dtype, device="cuda")
        self.vc = torch.zeros_like(self.kc)
        self.pages_ws = torch.zeros(sv.sv_pages_workspace_size(self.B, pages), dtype=torch.uint8, device="cuda")
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        self.freq = (10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) * 2 / R)).float().cuda()
        self.history = [[([], []) for _ in range(LAYERS)] for _ in range(self.B)]  # rows of k and v before the rotation
        self.prefill()
        # a step's inputs and outputs
        self.qkv = self.normal(LAYERS, self.B, HQ + 2 * HKV, D)
        self.out = torch.zeros((LAYERS, self.B, HQ, D), dtype=dtype, device="cuda")
        self.head = self.normal(V, HQ * D) * 0.2
        self.u = torch.zeros(self.B, device="cuda")
        self.logits = torch.zeros((self.B, V), dtype=dtype, device="cuda")
        self.tokens = dev([-7] * self.B)
        self.logprobs = torch.zeros(self.B, device="cuda")
        self.probs = torch.zeros((self.B, V), device="cuda")
        full = lambda x, t: torch.full((self.B,), x, dtype=t, device="cuda")  # noqa: E731
        self.settings = dict(temperature=full(SCALE, torch.float32), top_k=full(50, torch.int32), top_p=full(0.9, torch.float32))
        self.cu, self.target = dev(range(self.B + 1)), torch.zeros_like(self.ctx)
        self.cu_groups = dev(np.cumsum([0] + [len(r) for r in ROWS]).tolist())
        self.prefix = dev([n // 16 * 16 for n in PROMPTS])
        self.params = []
        for layer in range(LAYERS):
            p = sv.make_prefix_params(q=self.qkv[layer, :, :HQ], k_cache=self.kc[layer], v_cache=self.vc[layer],
                                      block_table=self.table, ctx_lens=self.ctx, cu_tokens=self.cu, cu_groups=self.cu_groups,
                                      prefix_lens=self.prefix, out=self.out[layer], max_tokens=1, max_group_tokens=self.B)
            if layer == 0:  # the layers run one after the other: one workspace
                self.attn_ws = torch.zeros(sv.sv_prefix_attention_workspace_size(p), dtype=torch.uint8, device="cuda")
            p.workspace, p.workspace_bytes = self.attn_ws.data_ptr(), self.attn_ws.numel()
            self.params.append(p)

    def reserve(self, target):
        sv.sv_pages_reserve(self.ctx, target, self.table, self.held, self.refs, self.src, self.dst, self.count,
                            workspace=self.pages_ws)
        sv.sv_pages_copy(self.kc, self.vc, self.src, self.dst, self.count, workspace=self.ws)

    def prefill(self):
        new = [0] * self.B
        for rows, n in zip(ROWS, PROMPTS):
            new[rows[0]] = n
        self.reserve(dev(new))
        cu = dev(np.cumsum([0] + new).tolist())
        for layer in range(LAYERS):
            k, v = self.normal(sum(new), HKV, D), self.normal(sum(new), HKV, D)
            sv.sv_rope_append(None, k, v, None, self.kc[layer], self.vc[layer], self.table, self.ctx, cu, self.freq,
                              new_ctx_lens=self.after, workspace=self.ws)
            for rows, n in zip(ROWS, PROMPTS):
                at = int(cu[rows[0]])
                for b in rows:
                    self.history[b][layer] = (list(k[at:at + n]), list(v[at:at + n]))
        self.ctx.copy_(self.after)
        parents, children = zip(*[(rows[0], b) for rows in ROWS for b in rows[1:]])
        sv.sv_pages_fork(dev(parents), dev(children), self.table, self.ctx, self.held, self.refs, workspace=self.pages_ws)

    def step(self):
        """What is captured: everything between the projections' inputs and the next tokens."""
        torch.add(self.ctx, 1, out=self.target)
        self.reserve(self.target)
        for layer in range(LAYERS):
            rows = self.qkv[layer]
            q = rows[:, :HQ]
            sv.sv_rope_append(q, rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:], q, self.kc[layer], self.vc[layer], self.table,
                              self.ctx, self.cu, self.freq, new_ctx_lens=self.after, workspace=self.ws)
            sv.sv_prefix_attention(self.params[layer])
        torch.matmul(self.out[-1].view(self.B, HQ * D), self.head.t(), out=self.logits)
        sv.sv_sample_tokens(self.logits, self.u, self.tokens, logprobs=self.logprobs, probs=self.probs, workspace=self.ws,
                            **self.settings)

    def errors(self):
        return [sv.sv_get_device_error(w) for w in (self.ws, self.attn_ws, self.pages_ws)]

    def state(self):
        return [self.table, self.held, self.ctx, self.refs, self.kc, self.vc]


def inputs_of(e, step):
    g = torch.Generator(device="cuda").manual_seed(100 + step)
    return (torch.randn(e.qkv.shape, generator=g, device="cuda").to(e.dtype),
            torch.rand(e.B, generator=g, device="cuda"))


def check_step(e, qkv):
    half = torch.finfo(e.dtype).eps / 2
    ctx = e.ctx.tolist()
    table = e.table.cpu().numpy()
    freq = e.freq.cpu().numpy()
    for layer in range(LAYERS):
        kc, vc = e.kc[layer].double().cpu().numpy(), e.vc[layer].double().cpu().numpy()
        want_q = oracle.rotate(qkv[layer, :, :HQ].double().cpu().numpy(), ctx, freq)
        q = e.qkv[layer, :, :HQ].double().cpu().numpy()     # rotated in place
        both = np.abs(qkv[layer, :, :HQ].double().cpu().numpy()).reshape(e.B, HQ, -1)
        size = np.zeros_like(both)
        size[..., :R // 2] = size[..., R // 2:R] = both[..., :R // 2] + both[..., R // 2:R]
        low = 2.0 ** -25 if e.dtype == torch.float16 else 0.0
        assert (np.abs(q - want_q) <= half * 1.0001 * np.abs(want_q) + 5e-7 * size + low).all()
        for b in range(e.B):
            k, v = e.history[b][layer]
            k.append(qkv[layer, b, HQ:HQ + HKV])
            v.append(qkv[layer, b, HQ + HKV:])
            n = ctx[b] + 1
            assert len(k) == n
            rows = torch.stack(k).double().cpu().numpy()
            want = oracle.rotate(rows, range(n), freq)
            size = np.zeros_like(want)
            size[..., :R // 2] = size[..., R // 2:R] = np.abs(rows[..., :R // 2]) + np.abs(rows[..., R // 2:R])
            at = [(table[b, i // 16], i % 16) for i in range(n)]
            got = np.stack([kc[page, :, slot] for page, slot in at])
            assert (np.abs(got - want) <= half * 1.0001 * np.abs(want) + 5e-7 * size + low).all(), (layer, b)
            got = np.stack([vc[page, :, slot] for page, slot in at])
            np.testing.assert_array_equal(got, torch.stack(v).double().cpu().numpy())
        want, _ = oracle.chunk_attention(q, kc, vc, table, ctx, range(e.B + 1))
        mean, _ = oracle.chunk_attention(q, kc, np.abs(vc), table, ctx, range(e.B + 1))
        tol = half * (mean + np.abs(want)) * 1.001 + 2e-4 * mean + low
        assert (np.abs(e.out[layer].double().cpu().numpy() - want) <= tol).all(), layer
    logits, probs = e.logits.double().cpu().numpy(), e.probs.double().cpu().numpy()
    for b in range(e.B):
        token, logprob, want, gap = oracle.sample_token(logits[b], float(e.u[b]), float(np.float32(SCALE)), 50,
                                                        float(np.float32(0.9)))
        assert gap > 1e-9 and int(e.tokens[b]) == token   # (these uniforms lie at no border)
        np.testing.assert_allclose(probs[b], want, rtol=2.0 ** -22 * 3, atol=1e-44)
        assert abs(float(e.logprobs[b]) - logprob) <= 2.0 ** -23 * (2 + 2 * abs(logprob))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_samples_of_shared_prompts(dtype):
    e = Engine(dtype)
    assert e.errors() == [0, 0, 0]
    start = [t.clone() for t in e.state()]
    tokens, outs = [], []
    for step in range(STEPS):
        qkv, u = inputs_of(e, step)
        e.qkv.copy_(qkv)
        e.u.copy_(u)
        e.step()
        assert e.errors() == [0, 0, 0]
        check_step(e, qkv)
        tokens.append(e.tokens.clone())
        outs.append(e.out.clone())
        e.ctx.copy_(e.after)
    assert e.ctx.tolist() == [n + STEPS for n, rows in zip(PROMPTS, ROWS) for _ in rows]
    assert len({tuple(t.tolist()) for t in tokens}) > 1
    # the same steps from a graph
    for t, x in zip(e.state(), start):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        e.step()
        e.ctx.copy_(e.after)
    for t, x in zip(e.state(), start):
        t.copy_(x)
    for step in range(STEPS):
        qkv, u = inputs_of(e, step)
        e.qkv.copy_(qkv)
        e.u.copy_(u)
        graph.replay()
        assert torch.equal(e.tokens, tokens[step]) and torch.equal(e.out, outs[step])
    assert e.errors() == [0, 0, 0]


def test_two_engines_at_once():
    """Two programs on two streams, each with its own state and workspaces."""
    engines, alone = [Engine(torch.bfloat16, seed) for seed in (1, 2)], []
    start = [[t.clone() for t in e.state()] for e in engines]
    for e in engines:
        got = []
        for step in range(6):
            qkv, u = inputs_of(e, step)
            e.qkv.copy_(qkv)
            e.u.copy_(u)
            e.step()
            e.ctx.copy_(e.after)
            got.append((e.tokens.clone(), e.out.clone()))
        alone.append(got)
    for e, s in zip(engines, start):
        for t, x in zip(e.state(), s):
            t.copy_(x)
    torch.cuda.synchronize()
    streams, both = [torch.cuda.Stream() for _ in engines], [[], []]
    for step in range(6):
        for e, stream, got in zip(engines, streams, both):
            with torch.cuda.stream(stream):
                qkv, u = inputs_of(e, step)
                e.qkv.copy_(qkv)
                e.u.copy_(u)
                e.step()
                e.ctx.copy_(e.after)
                got.append((e.tokens.clone(), e.out.clone()))
    torch.cuda.synchronize()
    for got, want in zip(both, alone):
        for (t, o), (tw, ow) in zip(got, want):
            assert torch.equal(t, tw) and torch.equal(o, ow)
