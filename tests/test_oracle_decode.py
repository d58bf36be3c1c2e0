"""Pins of the rotation and sampling oracles: complex numbers, closed forms, the
distribution that sampling must reproduce."""

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(0)
    x, freq = rng.standard_normal((3, 2, 24)), np.float32(10000.0) ** (-np.arange(8, dtype=np.float32) / 8)
    pos = [0, 1, 900001]
    got = oracle.rotate(x, pos, freq, interleaved, amplitude=1.25)
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    for t, p in enumerate(pos):
        z = 1.25 * (x[t, :, a] + 1j * x[t, :, b]) * np.exp(1j * p * freq.astype(np.float64))
        np.testing.assert_allclose(got[t, :, a], z.real, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(got[t, :, b], z.imag, rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(got[..., 16:], x[..., 16:])
    np.testing.assert_allclose(got[0, :, :16], 1.25 * x[0, :, :16], rtol=1e-15)


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    freq = np.float32(100.0) ** (-np.arange(8, dtype=np.float32) / 8)
    dots = [float((oracle.rotate(q, [p + 7], freq) * oracle.rotate(k, [p], freq)).sum()) for p in (0, 5, 1234)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_append_lands_in_the_slots():
    rng = np.random.default_rng(2)
    kc, vc = rng.standard_normal((4, 2, 4, 16)), rng.standard_normal((4, 2, 4, 16))
    q, k, v = rng.standard_normal((4, 2, 16)), rng.standard_normal((4, 2, 16)), rng.standard_normal((4, 2, 16))
    freq = np.ones(8, dtype=np.float32)
    out, k2, v2, lens = oracle.rope_append(q, k, v, kc, vc, [[2, 0], [1, 3]], [3, 5], [0, 2, 3], freq, page_size=4)
    assert lens.tolist() == [5, 6] and np.isnan(out[3]).all() and not np.isnan(out[:3]).any()
    np.testing.assert_array_equal(v2[2, :, 3], v[0])
    np.testing.assert_array_equal(v2[0, :, 0], v[1])
    np.testing.assert_array_equal(v2[3, :, 1], v[2])
    np.testing.assert_allclose(k2[3, :, 1], oracle.rotate(k[2:3], [5], freq)[0])
    changed = (v2 != vc).any(axis=(1, 3))
    assert changed.sum() == 3


def test_filters_by_hand():
    x = np.log([0.1, 0.4, 0.2, 0.2, 0.1])
    assert oracle.kept(x)[0] == [1, 2, 3, 0, 4]
    assert oracle.kept(x, top_k=2)[0] == [1, 2]
    assert oracle.kept(x, top_p=0.5)[0] == [1, 2]
    assert oracle.kept(x, top_p=0.61)[0] == [1, 2, 3]
    assert oracle.kept(x, top_k=2, top_p=0.65)[0] == [1]      # 0.4 of 0.6
    assert oracle.kept(x, top_p=0.0)[0] == [1] and oracle.kept(x, temperature=0)[0] == [1]
    assert oracle.kept(x, min_p=0.49)[0] == [1, 2, 3] and oracle.kept(x, min_p=1.5)[0] == [1]
    assert oracle.kept([1.0, 1.0, -np.inf, 1.0], top_k=2)[0] == [0, 1]
    token, logprob, probs, _ = oracle.sample_token(x, 0.55, top_p=0.61)
    assert token == 2 and np.isclose(logprob, np.log(0.25)) and np.allclose(probs, [0, 0.5, 0.25, 0.25, 0])


def test_draws_follow_the_shares():
    rng = np.random.default_rng(3)
    x = rng.standard_normal(40)
    _, _, probs, _ = oracle.sample_token(x, 0.0, temperature=0.7, top_k=12)
    drawn = [oracle.sample_token(x, u, temperature=0.7, top_k=12)[0] for u in (np.arange(4000) + 0.5) / 4000]
    share = np.bincount(drawn, minlength=40) / 4000
    np.testing.assert_allclose(share, probs, atol=1 / 4000)
