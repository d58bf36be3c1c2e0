"""The append with the position rotation on the GPU against the oracle.

Tolerance, element by element: the result is rounded once to 16 bits (half a step,
eps / 2 of it; below the smallest normal fp16 2^-25), from fp32 products of an
angle that is off by pi 2^-25 at most, cos and sin by two units in the last place
more: 5e-7 of |a| + |c| times the amplitude.  v and what does not turn are bit copies."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_sv_gb300 import binding as sv
from tests.gpu_support import ensure_lib

pytestmark = pytest.mark.gpu
PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


@pytest.fixture(scope="module", autouse=True)
def lib():
    ensure_lib()


def setup(lens, new, Hq, Hkv, D, dtype, page=16, fused=False, pad=0, spare=3, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(new) + pad
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    first = [n // page for n in lens]
    held = [-(-(a + b) // page) for a, b in zip(lens, new)]
    pages = sum(h - f for h, f in zip(held, first)) + spare
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    width = max(max(held), 1)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, (f, h) in enumerate(zip(first, held)):
        table[b, f:h] = torch.tensor(order[at:at + h - f], dtype=torch.int32)
        at += h - f
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    if fused:
        rows = normal(T, Hq + 2 * Hkv, D)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    else:
        q, k, v = normal(T, Hq, D), normal(T, Hkv, D), normal(T, Hkv, D)
    return dict(q=q, k=k, v=v, kc=normal(pages, Hkv, page, D), vc=normal(pages, Hkv, page, D), table=table.cuda(),
                ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=cu)


def frequencies(r, base=10000.0):
    return (base ** (-torch.arange(r // 2, dtype=torch.float64) * 2 / r)).float().cuda()


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, x, r, interleaved, amplitude, dtype):
    """got and want [..., D]; x: what was turned."""
    eps = torch.finfo(dtype).eps / 2
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    size = np.zeros_like(want)
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(amplitude)
    tol = eps * np.abs(want) * 1.0001 + 5e-7 * size + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    worst = np.max(np.abs(got - want) / np.maximum(tol, 1e-300)) if want.size else 0.0
    assert worst <= 1.0, worst
    np.testing.assert_array_equal(got[..., r:], want[..., r:])


def check(s, freq, interleaved=False, amplitude=1.0, positions=None, page=16, in_place=False):
    T, Hq, D = s["q"].shape
    r = 2 * freq.numel()
    want = oracle.rope_append(f64(s["q"]), f64(s["k"]), f64(s["v"]), f64(s["kc"]), f64(s["vc"]), s["table"].tolist(),
                              s["ctx"].tolist(), s["cu"].tolist(), freq.cpu().numpy(), interleaved=interleaved,
                              amplitude=amplitude, positions=None if positions is None else positions.tolist(),
                              page_size=page)
    q0, k0, kc, vc = s["q"].clone(), s["k"].clone(), s["kc"].clone(), s["vc"].clone()
    q = s["q"].clone() if in_place else s["q"]
    out = q if in_place else torch.full_like(q, 7.0)
    after = torch.zeros_like(s["ctx"])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.sv_rope_append(q, s["k"], s["v"], out, kc, vc, s["table"], s["ctx"], s["cu"], freq, positions=positions,
                      interleaved=interleaved, amplitude=amplitude, new_ctx_lens=after, workspace=ws)
    assert sv.sv_get_device_error(ws) == 0
    np.testing.assert_array_equal(after.cpu().numpy(), want[3])
    N = int(s["cu"][-1])
    close(f64(out[:N]), want[0][:N], f64(q0[:N]), r, interleaved, amplitude, q.dtype)
    if N < T:
        assert torch.equal(out[N:], q0[N:] if in_place else torch.full_like(out[N:], 7.0))
    np.testing.assert_array_equal(f64(vc), want[2])
    # the cache: what was not written is as it was, what was is near the oracle's
    turned = np.zeros(want[1].shape)
    pos_in_cache = np.zeros(want[1].shape[:1] + want[1].shape[2:3], dtype=bool)
    for b, L in enumerate(s["ctx"].tolist()):
        n0, n1 = int(s["cu"][b]), int(s["cu"][b + 1])
        for i in range(n1 - n0):
            at = int(s["table"][b, (L + i) // page]), (L + i) % page
            turned[at[0], :, at[1]] = f64(k0[n0 + i])
            pos_in_cache[at] = True
    got = f64(kc)
    written = np.broadcast_to(pos_in_cache[:, None, :], got.shape[:3])
    np.testing.assert_array_equal(got[~written], f64(s["kc"])[~written])
    close(got[written], want[1][written], turned[written], r, interleaved, amplitude, q.dtype)


CASES = [  # lens, new, Hq, Hkv, D, rotary
    ([511], [1], 8, 2, 64, 64),
    ([1000, 0, 15, 16, 1599], [1, 1, 1, 1, 1], 32, 8, 128, 128),
    ([0, 31, 100], [33, 0, 7], 12, 4, 64, 32),
    ([7] * 40, [1, 3] * 20, 4, 1, 128, 64),             # more than 32 sequences: the search
    ([0, 900001, 3], [5, 300, 800], 8, 8, 64, 64),      # long calls: four tokens per CTA, tokens not a multiple
    ([3, 77], [2, 9], 5, 1, 80, 48),                    # a head size without a kernel of its own
    ([20], [3], 2, 2, 16, 16),
    ([20, 5], [3, 1], 3, 3, 256, 256),
]


@pytest.mark.parametrize("lens,new,Hq,Hkv,D,r", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_against_the_oracle(lens, new, Hq, Hkv, D, r, dtype, interleaved):
    check(setup(lens, new, Hq, Hkv, D, dtype, seed=len(lens)), frequencies(r), interleaved)


def test_slices_of_the_fused_projection_padding_and_amplitude():
    for seed, pad in ((1, 0), (2, 5), (3, 1200)):
        s = setup([100, 0, 31], [17, 0, 2], 12, 4, 64, torch.bfloat16, fused=True, pad=pad, seed=seed)
        check(s, frequencies(64, 500000.0), amplitude=1.37)
        check(s, frequencies(32), interleaved=True, amplitude=-0.5)


def test_in_place_and_page_sizes():
    for page in (1, 8, 16, 48):
        s = setup([100, 0, 31], [17, 1, 2], 6, 2, 64, torch.float16, page=page, seed=page)
        check(s, frequencies(64), page=page, in_place=True)


def test_far_positions_and_positions_of_their_own():
    """Angles stay exact where fp32 products of position and frequency are off by whole radians."""
    g = torch.Generator().manual_seed(5)
    s = setup([2 ** 27 - 5, 10], [5, 40], 4, 2, 64, torch.float16, seed=9)
    check(s, frequencies(64, 1000000.0))
    pos = torch.randint(-2 ** 29, 2 ** 29, (45,), generator=g, dtype=torch.int32).cuda()
    pos[0], pos[1] = 0, -1
    check(s, frequencies(64), positions=pos)
    odd = torch.tensor([0.0, -1.0, 3.1415927, 1023.9, 2.0 ** -100, 1e-45, 0.1, 6.2831855], device="cuda")
    near = torch.randint(-2 ** 20, 2 ** 20, (45,), generator=g, dtype=torch.int32).cuda()
    check(s, odd, positions=near)


def test_frequencies_without_an_angle_give_nan():
    s = setup([4], [2], 2, 1, 64, torch.bfloat16)
    freq = torch.tensor([1.0, float("inf"), float("nan"), 1024.0, 0.5, 0, 0, 0], device="cuda")
    out = torch.empty_like(s["q"])
    sv.sv_rope_append(s["q"], s["k"], s["v"], out, s["kc"], s["vc"], s["table"], s["ctx"], s["cu"], freq)
    bad = out[..., :16].isnan().all(0).all(0).nonzero().flatten().tolist()
    assert bad == [1, 2, 3, 9, 10, 11] and not out[..., 16:].isnan().any()


def test_without_q_and_without_tokens():
    s = setup([4, 30], [2, 3], 2, 2, 64, torch.bfloat16)
    freq = frequencies(64)
    kc, vc = s["kc"].clone(), s["vc"].clone()
    sv.sv_rope_append(None, s["k"], s["v"], None, kc, vc, s["table"], s["ctx"], s["cu"], freq)
    out = torch.empty_like(s["q"])
    kc2, vc2 = s["kc"].clone(), s["vc"].clone()
    sv.sv_rope_append(s["q"], s["k"], s["v"], out, kc2, vc2, s["table"], s["ctx"], s["cu"], freq)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and not torch.equal(kc, s["kc"])
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    after = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    sv.sv_rope_append(none, none, none, none, kc, vc, s["table"], s["ctx"], cu, freq, new_ctx_lens=after)
    assert after.tolist() == [4, 30] and torch.equal(kc, kc2)


def test_leaves_out_what_does_not_fit():
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.ones((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(k, 7.0)
    freq = frequencies(32)
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    after = torch.zeros(2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([30, 2], dtype=torch.int32, device="cuda")  # 30 + 4 > 2 pages
    sv.sv_rope_append(k, k, k, out, kc, vc, table, lens, cu, freq, new_ctx_lens=after, workspace=ws)
    assert sv.sv_get_device_error(ws) == sv.SV_DEVERR_BAD_LENGTH
    assert after.tolist() == [30, 4] and vc[:2].abs().sum() == 0 and vc[2, :, 2:4].eq(1).all() and vc.sum() == 256
    assert out[:4].eq(7).all() and not out[4:].eq(7).any()
    lens = torch.tensor([0, 15], dtype=torch.int32, device="cuda")  # slot 16 lies in page 9 of 4
    sv.sv_rope_append(k, k, k, out, kc, vc, table, lens, cu, freq, new_ctx_lens=after, workspace=ws)
    assert sv.sv_get_device_error(ws) == sv.SV_DEVERR_BAD_PAGE
    assert vc[2, :, 15].eq(1).all() and vc[0, :, :4].eq(1).all() and vc[3].abs().sum() == 0
    assert not out.eq(7).any()
    # lengths past the token rows, and a negative one
    for bad_cu, bad_len in (([0, 4, 7], [0, 0]), ([0, 4, 2], [0, 0]), ([0, 4, 6], [0, -1])):
        sv.sv_rope_append(k, k, k, out, kc, vc, table, torch.tensor(bad_len, dtype=torch.int32, device="cuda"),
                          torch.tensor(bad_cu, dtype=torch.int32, device="cuda"), freq, workspace=ws)
        assert sv.sv_get_device_error(ws) == sv.SV_DEVERR_BAD_LENGTH


def test_captured_and_replayed_on_another_stream():
    s = setup([100, 0, 31], [17, 1, 2], 6, 2, 64, torch.bfloat16)
    freq = frequencies(64)
    out, after = torch.empty_like(s["q"]), torch.zeros_like(s["ctx"])
    kc, vc = s["kc"].clone(), s["vc"].clone()
    call = lambda o, a, b: sv.sv_rope_append(s["q"], s["k"], s["v"], o, a, b, s["table"], s["ctx"], s["cu"], freq,  # noqa: E731
                                             new_ctx_lens=after)
    call(out, kc, vc)
    torch.cuda.synchronize()
    out2, kc2, vc2 = torch.empty_like(out), s["kc"].clone(), s["vc"].clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call(out2, kc2, vc2)
        graph.replay()
        s["q"].add_(1)
        graph.replay()
    side.synchronize()
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and not torch.equal(out, out2)
    call(out, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


@pytest.mark.parametrize("f", [float(np.nextafter(np.float32(1024), np.float32(0))), 700.1, 1.0, 0.7654321])
def test_angles_at_the_ends_of_both_ranges(f):
    """Angles within 2^-24 of half a turn at positions next to 2^31, where they show: next to a quarter turn the cosine
    (the pair (1, 0) turned) is small, so its 16 bits hold the angle's error.  Beside that the cosine is off by
    fp32's rounding of it and half a step of bf16, relative."""
    exact = Fraction(float(np.float32(f))) / (2 * PI)                # turns per position
    step = np.uint64(int(exact * 2 ** 64) % 2 ** 64)                 # 2^-33 of a turn off at most at 2^31
    x = np.arange(2 ** 31 - 2 ** 22, 2 ** 31, dtype=np.uint64)
    half_turns = (x * step).view(np.int64).astype(np.float64) / 2 ** 63
    x = x[np.argsort(np.abs(np.abs(half_turns) - 0.5))[:24]].astype(np.int64)
    x = np.concatenate([x, -x])
    T = len(x)
    q = torch.zeros((T, 1, 16), dtype=torch.bfloat16, device="cuda")
    q[:, :, :8] = 1.0
    out, cache = torch.empty_like(q), torch.zeros((T, 1, 1, 16), dtype=torch.bfloat16, device="cuda")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    sv.sv_rope_append(q, q, q, out, cache, cache.clone(), ints(list(range(T)))[None], ints([0]), ints([0, T]),
                      torch.full((8,), f, device="cuda"), positions=ints(x))
    for t in range(T):
        turns = exact * int(x[t]) % 1
        want = float(np.sin(float(2 * PI * (Fraction(1, 4) - turns if turns < Fraction(1, 2) else turns - Fraction(3, 4)))))
        assert abs(want) < 1e-4
        assert (out[t, 0, :8].double() - want).abs().max() <= np.pi * 2.0 ** -24 + 1.01 * 2.0 ** -8 * abs(want), int(x[t])


def test_cache_offsets_past_32_bits():
    """The last pages of a pool of 2.6e9 elements, from token rows whose offsets pass 2^31 too."""
    pages, T = 40000, 3
    kc, vc = (torch.zeros((pages, 8, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wide = torch.empty((T, 1 << 30), dtype=torch.bfloat16, device="cuda")
    k = wide[:, :1024].view(T, 8, 128)
    k.copy_(torch.randn((T, 8, 128), device="cuda"))
    out = torch.empty_like(k, memory_format=torch.contiguous_format)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sv.sv_rope_append(k, k, k, out, kc, vc, ints([[0, pages - 1], [pages - 2, 1]]), ints([63, 10]), ints([0, 2, 3]), frequencies(64),
                      workspace=ws)
    assert sv.sv_get_device_error(ws) == 0
    assert torch.equal(vc[0, :, 63], k[0]) and torch.equal(vc[pages - 1, :, 0], k[1]) and torch.equal(vc[pages - 2, :, 10], k[2])
    want = oracle.rotate(f64(k), [63, 64, 10], frequencies(64).cpu().numpy())
    close(f64(out), want, f64(k), 64, False, 1.0, torch.bfloat16)
    for t, at in enumerate([(0, 63), (pages - 1, 0), (pages - 2, 10)]):
        assert torch.equal(kc[at[0], :, at[1]], out[t])
    assert int(kc.any(dim=3).any(dim=1).sum()) == 3


def test_many_sequences():
    """More sequences than a search takes in three rounds, and than the grid has threads, most without a token."""
    B = 70000
    new = torch.zeros(B, dtype=torch.int64)
    new[torch.tensor([0, 5, 6, 40000, 65536, B - 1])] = torch.tensor([2, 1, 3, 1, 2, 4])
    T = int(new.sum())
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).int().cuda()
    ctx = (torch.arange(B, dtype=torch.int32) % 29).cuda()
    table = torch.arange(2 * B, dtype=torch.int32).view(B, 2).cuda()
    k = torch.randn((T, 1, 16), device="cuda").half()
    kc, vc = (torch.zeros((2 * B, 1, 16, 16), dtype=torch.float16, device="cuda") for _ in range(2))
    after = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    sv.sv_rope_append(None, k, k, None, kc, vc, table, ctx, cu, frequencies(16), new_ctx_lens=after)
    assert torch.equal(after, ctx + new.int().cuda())
    seen = 0
    for b in new.nonzero().flatten().tolist():
        for i in range(int(new[b])):
            slot = int(ctx[b]) + i
            assert torch.equal(vc[2 * b + slot // 16, :, slot % 16], k[seen])
            seen += 1
    assert int(vc.any(dim=3).sum()) == T
