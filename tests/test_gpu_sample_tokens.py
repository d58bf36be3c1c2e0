"""Token sampling on the GPU against the oracle: tokens are equal, kept sets are
equal, logprobs and probabilities within fp32.

The kernel's weights are off by 2^-36 of the largest, its sums of them are exact (in
practice off by less than 2^-30 of the row), so a
token may differ from float64's only where the uniform (or a filter's limit) lies
within that of a border of sums: a draw nearer than 1e-9 to one (a uniform of one half
over a symmetric row) may take the entry on either side.
Logprobs: the logarithm's argument is off by 2^-23 at most, and so are the
exponent's product and its sum, each at most 2^-23 of |logprob| more.
Probabilities: the hardware's power 2^-22, a quotient and two products 2^-23 each."""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def lib():
    ensure_lib()


def sample(logits, u, probs=False, workspace=None, **settings):
    R, V = logits.shape
    put = lambda v, t: None if v is None else torch.tensor(np.broadcast_to(v, R).copy(), dtype=t, device="cuda")  # noqa: E731
    tokens = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    logprobs = torch.full((R,), 7.0, device="cuda")
    rows = torch.full((R, V), 7.0, device="cuda") if probs else None
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.sv_sample_tokens(logits, u, tokens, temperature=put(settings.get("temperature"), torch.float32),
                        top_k=put(settings.get("top_k"), torch.int32), top_p=put(settings.get("top_p"), torch.float32),
                        min_p=put(settings.get("min_p"), torch.float32), logprobs=logprobs, probs=rows, workspace=ws)
    return tokens, logprobs, rows, sv.sv_get_device_error(ws)


def check(logits, u, near=1e-9, **settings):
    tokens, logprobs, probs, err = sample(logits, u, probs=True, **settings)
    assert err == 0
    values, probs = logits.double().cpu().numpy(), probs.double().cpu().numpy()
    R = len(values)
    f32 = lambda k, d: np.broadcast_to(np.float32(settings.get(k, d) if settings.get(k) is not None else d), R)  # noqa: E731
    top_k = np.broadcast_to(settings.get("top_k") if settings.get("top_k") is not None else 0, R)
    for r in range(R):
        draw = lambda x: oracle.sample_token(values[r], x, float(f32("temperature", 1.0)[r]), int(top_k[r]),  # noqa: E731
                                             float(f32("top_p", 1.0)[r]), float(f32("min_p", 0.0)[r]))
        token, logprob, want, gap = draw(float(u[r]))
        if gap <= near and tokens[r] != token:
            token, logprob = next(d[:2] for d in (draw(float(u[r]) - near), draw(float(u[r]) + near)) if d[0] != token)
        assert tokens[r] == token, (r, gap)
        assert not probs[r][want == 0].any() and probs[r][want > 1e-37].all()  # (between them: what fp32 can hold)
        np.testing.assert_allclose(probs[r], want, rtol=2.0 ** -22 * 3, atol=1e-44)
        assert abs(float(logprobs[r]) - logprob) <= 2.0 ** -23 * (2 + 2 * abs(logprob)), (float(logprobs[r]), logprob)


def random_logits(R, V, dtype, seed, sigma=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = sigma * torch.randn((R, V), generator=g, device="cuda")
    x[:, : max(1, V // 50)] += 10 * torch.rand((R, max(1, V // 50)), generator=g, device="cuda")
    return x[:, torch.randperm(V, generator=g, device="cuda")].to(dtype), torch.rand(R, generator=g, device="cuda")


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.05),
            dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02), dict(temperature=1.3, top_k=7, top_p=0.5),
            dict(temperature=0.0), dict(top_p=0.0), dict(top_p=1.0, top_k=-1, min_p=0.0), dict(top_k=10 ** 9, top_p=0.3),
            dict(min_p=1.0), dict(min_p=2.0), dict(temperature=0.05, top_p=0.999), dict(temperature=20.0, top_p=0.6)]


@pytest.mark.parametrize("V", [1, 2, 7, 31, 1000, 2049, 5003])
@pytest.mark.parametrize("dtype", TYPES)
def test_small_vocabularies(V, dtype):
    for i, settings in enumerate(SETTINGS):
        check(*random_logits(3, V, dtype, seed=V + i), **settings)


@pytest.mark.parametrize("V,R,dtype", [(32000, 2, torch.float32), (50257, 2, torch.bfloat16), (128256, 2, torch.float32),
                                       (151936, 1, torch.float16), (262144, 1, torch.float32)])
def test_large_vocabularies(V, R, dtype):
    for i, settings in enumerate([dict(), dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02), dict(top_p=0.9),
                                  dict(temperature=1.5, top_k=5000, top_p=0.8), dict(temperature=8.0, top_p=0.7)]):
        check(*random_logits(R, V, dtype, seed=V + i), **settings)


@pytest.mark.parametrize("R", [5, 70, 300])
def test_batches_with_settings_of_their_own(R):
    """Rows of every kind in one call, in clusters of every size (few and many rows)."""
    rng = np.random.default_rng(R)
    logits, u = random_logits(R, 4111, torch.bfloat16, seed=R)
    check(logits, u, temperature=rng.choice([0.0, 0.5, 1.0, 1.5], R).astype(np.float32),
          top_k=rng.choice([0, 1, 5, 200, 3000, 9999], R), top_p=rng.choice([0.0, 0.5, 0.9, 1.0], R).astype(np.float32),
          min_p=rng.choice([0.0, 0.0, 0.1], R).astype(np.float32))


@pytest.mark.parametrize("dtype", TYPES)
def test_many_equal_logits(dtype):
    """More equal entries than are sorted at once: the threshold is found by the bits of their indices."""
    for V in (9000, 40000):
        x = torch.zeros((4, V), dtype=dtype, device="cuda")
        x[1, ::3] = 2.0
        x[2, ::2] = -1.0
        x[3] = torch.arange(V, device="cuda").remainder(5).to(dtype)
        u = torch.tensor([0.3, 0.77, 0.5, 0.999], device="cuda")
        for settings in (dict(), dict(top_k=V // 2 + 3), dict(top_p=0.40005), dict(top_k=V // 3, top_p=0.750003),
                         dict(top_k=5), dict(top_p=0.00011)):
            check(x, u, **settings)


def test_dense_bins_are_split_by_the_logits_bits():
    """Thousands of different logits within 1/32 of a power of two of each other."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = 5.0 + 0.01 * torch.rand((2, 20000), generator=g, device="cuda")
    x[1, 7] = 30.0
    x[1] -= 17.0
    for settings in (dict(top_k=7000), dict(top_p=0.613), dict(top_k=15000, top_p=0.5), dict(top_p=0.6, temperature=9.0)):
        check(x, torch.tensor([0.21, 0.87], device="cuda"), **settings)


def test_masked_entries_and_extreme_values():
    x = torch.full((6, 3001), -torch.inf, device="cuda")
    x[0, 17] = -3.0e38                                      # one entry
    x[1, [5, 2000]] = torch.tensor([1.0, 1.0], device="cuda")
    x[2, 100:200] = torch.linspace(-1e30, 1e30, 100, device="cuda")
    x[3, ::2] = 0.0
    x[3, 1::2] = -0.0                                       # equal to 0: lower indices first
    x[4, :50] = 3.0e38
    x[4, 50:90] = -3.0e38
    x[5, 2999:] = torch.tensor([1e-40, -1e-40], device="cuda")
    u = torch.tensor([0.9, 0.6, 0.2, 0.1, 0.5, 0.25], device="cuda")
    for settings in (dict(), dict(top_k=2), dict(top_p=0.5001), dict(min_p=0.3), dict(temperature=0.0), dict(top_k=1500)):
        check(x, u, **settings)


@pytest.mark.parametrize("settings", [dict(), dict(top_p=0.95, temperature=1.3), dict(top_p=0.98, min_p=0.02, temperature=1.2),
                                      dict(top_k=700), dict(top_k=1000, top_p=0.9), dict(top_p=0.995, temperature=1.2)])
def test_batches_that_give_a_cta_a_whole_row(settings):
    """More rows than SMs: runs of more entries than are summed in fp32, and flat rows whose nucleus is thousands of
    entries; a few rows against the oracle."""
    x, u = random_logits(160, 38000, torch.bfloat16, seed=21, sigma=2.0)
    some = [0, 77, 159]
    tokens, logprobs, probs, err = sample(x, u, probs=True, **settings)
    assert err == 0
    few = sample(x[some].contiguous(), u[some].contiguous(), probs=True, **settings)  # three rows: eight CTAs each
    for i, r in enumerate(some):
        args = [float(np.float32(settings.get(k, d))) for k, d in (("top_p", 1.0), ("min_p", 0.0))]
        token, logprob, want, gap = oracle.sample_token(x[r].double().cpu().numpy(), float(u[r]),
                                                        float(np.float32(settings.get("temperature", 1.0))),
                                                        settings.get("top_k", 0), *args)
        assert gap > 1e-9   # (these uniforms lie at no border)
        for t, lp, p in ((tokens[r], logprobs[r], probs[r]), (few[0][i], few[1][i], few[2][i])):
            assert int(t) == token
            assert abs(float(lp) - logprob) <= 2.0 ** -23 * (2 + 2 * abs(logprob))
            got = p.double().cpu().numpy()
            assert ((got > 0) == (want > 0)).all()
            np.testing.assert_allclose(got, want, rtol=2.0 ** -22 * 3, atol=1e-44)


def test_uniform_at_the_ends():
    x = torch.zeros((3, 1024), device="cuda")
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5], device="cuda")
    assert sample(x, u)[0].tolist() == [0, 1023, 512]
    x[:, :100] = x[:, 900:] = -torch.inf
    assert sample(x, u)[0].tolist() == [100, 899, 500]
    assert sample(x, u, top_k=10)[0].tolist() == [100, 109, 105]


def test_rows_without_a_token():
    x = torch.zeros((9, 500), device="cuda")
    x[0] = -torch.inf
    x[1, 3] = torch.inf
    x[2, 499] = torch.nan
    u = torch.full((9,), 0.5, device="cuda")
    u[3], u[4], u[5] = 1.0, -0.1, torch.nan
    t = np.ones(9, dtype=np.float32)
    t[6], t[7] = -1.0, np.inf
    tokens, logprobs, probs, err = sample(x, u, probs=True, temperature=t)
    assert err == sv.SV_DEVERR_BAD_VALUE
    assert tokens.tolist() == [-1] * 8 + [250]
    assert logprobs[:8].isnan().all() and probs[:8].isnan().all() and not probs[8].isnan().any()
    for name in ("top_p", "min_p", "temperature"):
        assert sample(x[8:], u[8:], **{name: np.float32("nan")})[0].tolist() == [-1]


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_at_any_stride_and_address(dtype):
    """Slices of a wider matrix: rows that start at every place within 16 bytes."""
    base, u = random_logits(8, 3100, dtype, seed=5)
    for off, V in ((0, 3100), (1, 3000), (3, 3001), (7, 2999), (8, 77), (5, 3)):
        x = base[:, off:off + V]
        check(x, u, top_k=30)
        check(x, u)


def test_probabilities_of_wider_rows_leave_the_rest():
    x, u = random_logits(3, 1000, torch.float32, seed=8)
    wide = torch.full((3, 1010), 7.0, device="cuda")
    tokens = torch.empty(3, dtype=torch.int32, device="cuda")
    sv.sv_sample_tokens(x, u, tokens, probs=wide[:, 3:1003])
    assert wide[:, :3].eq(7).all() and wide[:, 1003:].eq(7).all()
    assert (wide[:, 3:1003].sum(1) - 1).abs().max() < 1e-5


def test_same_tokens_on_every_run_and_stream():
    x, u = random_logits(64, 128256, torch.float32, seed=11)
    first = sample(x, u, top_p=0.9)[:2]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            again = sample(x, u, top_p=0.9)[:2]
        torch.cuda.synchronize()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured_and_replayed():
    x, u = random_logits(4, 5000, torch.bfloat16, seed=12)
    tokens = torch.empty(4, dtype=torch.int32, device="cuda")
    k = torch.full((4,), 20, dtype=torch.int32, device="cuda")
    sv.sv_sample_tokens(x, u, tokens, top_k=k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_sample_tokens(x, u, tokens, top_k=k)
    x.copy_(random_logits(4, 5000, torch.bfloat16, seed=13)[0])
    graph.replay()
    assert torch.equal(tokens, sample(x, u, top_k=20)[0])


def test_draft_tokens_and_distributions_feed_stochastic_acceptance():
    """A root and two children drawn from a draft's filtered distribution: with the target's logits equal to the draft's
    and no filter, the first child is accepted whatever its uniform."""
    V = 2000
    x, _ = random_logits(1, V, torch.float32, seed=14)
    draft = torch.empty((3, V), device="cuda")
    kids = torch.empty(2, dtype=torch.int32, device="cuda")
    u = torch.tensor([0.3, 0.8], device="cuda")
    sv.sv_sample_tokens(x.expand(2, V).contiguous(), u, kids, probs=draft[:2])
    tokens = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), kids])
    parents = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    child, length, bonus = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (3, 1, 1))
    nodes = torch.empty((1, 2), dtype=torch.int32, device="cuda")
    ws = torch.zeros(sv.sv_sample_accept_workspace_size(1, 3), dtype=torch.uint8, device="cuda")
    draft[2] = draft[0]
    sv.sv_sample_accept(x.expand(3, V).contiguous(), draft, V, 1.0, tokens, parents, cu, 1, 3, 3, 1,
                        torch.full((3,), 0.9999, device="cuda"), torch.full((3,), 0.5, device="cuda"), child, length, nodes,
                        bonus, ws)
    assert sv.sv_get_device_error(ws) == 0
    assert length.item() == 1 and nodes.tolist() == [[0, 1]]


@pytest.mark.parametrize("R", [3, 20, 50, 100, 170])
@pytest.mark.parametrize("V", [2049, 16395, 20011])
def test_clusters_whose_threads_have_unequal_parts(R, V):
    """Clusters of eight, four, two and one CTAs whose threads leave the loops over their parts one by one, before the
    barriers that follow; three rows against the oracle, and the same bits again."""
    base, u = random_logits(R, V + 3, torch.bfloat16, seed=R + V)
    x = base[:, 3:]
    for settings in (dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.95), dict(top_k=900)):
        tokens, logprobs, probs, err = sample(x, u, probs=True, **settings)
        again = sample(x, u, probs=True, **settings)
        assert err == 0 and again[3] == 0
        assert torch.equal(tokens, again[0]) and torch.equal(logprobs, again[1]) and torch.equal(probs, again[2])
        for r in (0, R // 2, R - 1):
            token, logprob, want, gap = oracle.sample_token(x[r].double().cpu().numpy(), float(u[r]), 1.0,
                                                            settings.get("top_k", 0), float(np.float32(settings.get("top_p", 1.0))))
            assert gap > 1e-9 and int(tokens[r]) == token
            assert ((probs[r] > 0).cpu().numpy() == (want > 0)).all()



def last_entry_rows():
    x = torch.full((2, 1 << 18), -1000.0, device="cuda")
    x[:, 0], x[:, 1], x[:, -1], x[:, 7] = 0.0, -0.5, -40.0, -41.0
    x[1, 3:260] = -2.0
    return x, torch.tensor([0.7, 0.999], device="cuda")


def test_the_last_entry_of_the_largest_vocabulary():
    """It may be kept with a weight below the last bit of the sums, in front of another such entry."""
    for settings in (dict(top_k=3), dict(top_k=4), dict(top_k=262)):
        check(*last_entry_rows(), **settings)


def test_min_p_below_the_last_bit_of_the_sums():
    """Entries that weigh as much are kept, and have their share, though no uniform draws them."""
    for settings in (dict(min_p=1e-30), dict(min_p=1e-30, top_k=262), dict(min_p=3e-18, top_k=500), dict(min_p=3e-18),
                     dict(min_p=1e-30, top_k=2000, temperature=0.7), dict(min_p=1e-30, top_p=0.9999)):
        check(*last_entry_rows(), **settings)
    x, u = random_logits(3, 3001, torch.float32, seed=17)
    x[:, 500:] -= 30.0
    for min_p in (1e-17, 1e-20, 1e-37):
        check(x, u, min_p=min_p)
        check(x, u, min_p=min_p, top_k=3000)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [4096, 20000])
def test_an_entry_without_weight_is_drawn_at_no_border(V, dtype):
    """Every run of eight holds seven weights a little below 2^-13 and then a mask of finite value; uniforms at the borders
    between them, within a few units of fp32 on either side."""
    rng = np.random.default_rng(V)
    R = 600
    x = torch.from_numpy(rng.uniform(-12.0, -9.1, (R, V)).astype(np.float32))
    x[:, 7::8] = -3.0e4
    x[:, -1] = 0.0
    x = x.to(dtype).cuda()
    w = x.double().exp()
    w[:, 7::8] = 0.0
    w[:, -1] = 1.0
    share = w.cumsum(1) / w.sum(1, keepdim=True)
    r = torch.arange(R)
    for run in (0, 3, 17):
        border = share[r, 8 * run + 6].float()
        for off in (-2, -1, 0, 1, 2):
            u = (border.view(torch.int32) + off).view(torch.float32)
            tokens, logprobs, _, err = sample(x, u)
            assert err == 0
            assert (x[r, tokens.long()] > -100).all() and (logprobs > -100).all()
            assert ((tokens == 8 * run + 6) | (tokens == 8 * run + 8)).all()


@pytest.mark.parametrize("settings", [dict(), dict(top_k=700), dict(top_k=300, top_p=0.9), dict(top_p=0.9), dict(min_p=1e-5)])
def test_the_batch_does_not_show_in_a_row(settings):
    """Flat rows with uniforms next to borders of their sums, alone and in batches of other sizes, which divide a row
    otherwise: the same bits."""
    g = torch.Generator(device="cuda").manual_seed(31)
    R, V = 400, 20011
    x = torch.rand((R, V), generator=g, device="cuda") - 10.5   # weights near 2^-14 of the largest
    x[:, 9000] = 0.0
    share = x.double().softmax(1).cumsum(1)
    u = share.gather(1, torch.randint(V // 4, V, (R, 1), generator=g, device="cuda"))[:, 0].float().clamp(max=1 - 2.0 ** -24)
    whole = sample(x, u, probs=True, **settings)
    assert whole[3] == 0
    for size in (1, 5, 40, 130):
        for at in range(0, 130 if size == 1 else R - size + 1, size):
            part = sample(x[at:at + size], u[at:at + size], probs=True, **settings)
            for a, b in zip(whole, part[:3]):
                assert torch.equal(a[at:at + size], b), (size, at)


@pytest.mark.parametrize("dtype", TYPES)
def test_the_batch_does_not_show_in_rows_of_every_kind(dtype):
    rng = np.random.default_rng(5)
    R, V = 320, 20011
    x, u = random_logits(R, V, dtype, seed=41, sigma=1.5)
    x[::7] *= 0.1                                               # flat ones
    x[3::11, ::2] = torch.finfo(dtype).min                      # masked by the type's lowest value
    x[5::13, 1::2] = -torch.inf
    settings = dict(temperature=rng.choice([0.0, 0.3, 1.0, 2.0], R).astype(np.float32),
                    top_k=rng.choice([0, 0, 1, 60, 513, 900, 3000, 99999], R),
                    top_p=rng.choice([0.0, 0.3, 0.9, 0.99999994, 1.0], R).astype(np.float32),
                    min_p=rng.choice([0.0, 0.0, 1e-30, 1e-4, 0.1], R).astype(np.float32))
    whole = sample(x, u, probs=True, **settings)
    assert whole[3] == 0
    for size in (1, 6, 45, 160):
        for at in range(0, 160 if size == 1 else R - size + 1, size):
            part = sample(x[at:at + size], u[at:at + size], probs=True, **{k: v[at:at + size] for k, v in settings.items()})
            for a, b in zip(whole, part[:3]):
                assert torch.equal(a[at:at + size], b), (size, at)


def test_settings_at_the_ends_of_their_types():
    x, u = random_logits(3, 5003, torch.float32, seed=51)
    for top_k in (2 ** 31 - 1, -2 ** 31, 2 ** 31 - 8):
        check(x, u, top_k=top_k)
        check(x, u, top_k=top_k, top_p=0.7)
    for temperature in (1e-45, 1e-38, 1e-30, 1e20, 1e30, 3.4e38):
        check(x, u, temperature=temperature)
        check(x, u, temperature=temperature, top_k=30, top_p=0.6)
        check(x, u, temperature=temperature, top_p=0.5)


@pytest.mark.parametrize("dtype", TYPES)
def test_small_min_p_keeps_by_relative_weight(dtype):
    """Weights next to a limit of a few units of the sums' last bit: what is kept is decided to 2^-22 of the weight (these
    random weights lie further from the limit)."""
    x, u = random_logits(4, 20011, dtype, seed=61, sigma=6.0)
    x[2, 3000:] -= 25.0
    for min_p in (2e-16, 1e-14, 1e-13, 1e-12, 3e-11, 1e-8, 1e-6, 5e-5, 7e-5):
        for settings in (dict(), dict(top_k=300), dict(top_k=9000)):
            check(x, u, min_p=min_p, **settings)


def test_offsets_past_32_bits():
    """The last rows of 2.2e9 logits, and of as many probabilities."""
    R, V = 17000, 131072
    x = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
    last, u = random_logits(3, V, torch.bfloat16, seed=71)
    x[-3:] = last
    every = torch.full((R,), 0.25, device="cuda")
    every[-3:] = u
    tokens, logprobs, probs, err = sample(x, every, probs=True, top_k=40)
    assert err == 0
    for a, b in zip((tokens, logprobs, probs), sample(last, u, probs=True, top_k=40)):
        assert torch.equal(a[-3:], b)
    assert tokens[:-3].eq(10).all() and probs[-4, :40].eq(0.025).all() and not probs[-4, 40:].any()


def test_many_small_rows():
    R, V = 100000, 33
    x, u = random_logits(R, V, torch.float32, seed=72)
    tokens, logprobs, _, err = sample(x, u)
    assert err == 0
    share = x.double().softmax(1)
    running = share.cumsum(1)
    gap = (running - u.double()[:, None]).abs().min(1).values
    want = (running <= u.double()[:, None]).sum(1)
    assert ((tokens == want) | (gap < 1e-9)).all() and (gap < 1e-9).sum() < 10
    got = share.log().gather(1, tokens.long()[:, None])[:, 0]
    assert ((logprobs - got).abs() <= 2.0 ** -23 * (2 + 2 * got.abs())).all()
