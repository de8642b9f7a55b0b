"""Pins of the training-step oracle: brute force, closed forms, difference quotients."""
import math

import numpy as np
import pytest

from oracle import training_oracle as T


@pytest.mark.parametrize("top", [127, 255])
def test_adam8_code_is_the_nearest_square(top):
    rng = np.random.default_rng(1)
    x = rng.standard_normal(BLOCKS := 256 * 3) * np.exp(3 * rng.standard_normal(BLOCKS))
    x = x.astype(np.float32).astype(np.float64)
    if top == 255:
        x = np.abs(x)
    k, d = T.adam8_encode(x, top)
    sq = np.arange(top + 1, dtype=np.float64) ** 2
    for b in range(3):
        y = T.rn32(np.abs(x[256 * b:256 * b + 256]) * T.rn32(1.0 / np.float64(d[b])))
        brute = np.array([int(np.argmin(np.abs(v - sq))) for v in y])       # argmin takes the lower index on a tie
        assert np.array_equal(np.abs(k[256 * b:256 * b + 256]), brute)
    assert np.abs(k).reshape(3, 256).max(axis=1).tolist() == [top] * 3      # the largest value takes the top code
    assert np.array_equal(np.sign(k)[k != 0], np.sign(x)[k != 0])


def test_adam8_ties_and_borders():
    # d = 1: the block's largest value is top^2, so y = |x| exactly
    top = 127
    j = np.arange(60, dtype=np.float64)
    mid = j * j + j + 0.5
    for shift, want in ((0.0, j), (2.0 ** -9, j + 1), (-(2.0 ** -9), j)):
        x = np.concatenate([mid + shift, [top * top]])
        k, d = T.adam8_encode(x, top)
        assert d[0] == 1.0 and np.array_equal(k[:-1], want)


def test_adam8_error_is_at_most_half_a_step():
    rng = np.random.default_rng(2)
    x = rng.standard_normal(1000).astype(np.float32).astype(np.float64)
    k, d = T.adam8_encode(x, 127)
    got = T.adam8_decode(k, d)
    step = np.repeat(d.astype(np.float64), 256)[:1000]
    # neighbours k^2 and (k + 1)^2 lie 2 k + 1 steps apart: the nearer one is within k + 1/2 of y
    assert (np.abs(got - x) <= (np.abs(k) + 0.5) * step * (1 + 1e-5)).all()


def test_adam8_special_blocks():
    x = np.zeros(256 * 4)
    x[256 + 7] = np.nan
    x[512 + 9] = np.inf
    x[768:] = 1e-40
    k, d = T.adam8_encode(x, 127)
    assert not k.any() and d[0] == 0 and np.isnan(d[1]) and np.isnan(d[2]) and d[3] == 0
    back = T.adam8_decode(k, d)
    assert not back[:256].any() and np.isnan(back[256:768]).all() and not back[768:].any()


def test_adamw_first_step_moves_by_the_sign():
    # t = 1 from zero states: m^ = g and v^ = g^2, so the update is g / (|g| + eps)
    g = np.array([3.0, -0.25, 1e-3, 0.0])
    m, v, _ = T.adamw_moments(g, None, np.zeros(4), np.zeros(4), 0.9, 0.999)
    p, u = T.adamw_param(np.ones(4), m, v, 1, 0.1, 0.0, 0.9, 0.999, 1e-8)
    assert np.allclose(u, [1, -1, 1, 0], atol=2e-5) and np.allclose(p, 1 - 0.1 * np.array([1, -1, 1, 0]), atol=2e-6)


def test_adamw_decay_shrinks_by_the_factor():
    p, _ = T.adamw_param(np.array([2.0]), np.zeros(1), np.zeros(1), 5, 0.1, 0.5, 0.9, 0.999, 1e-8)
    assert p[0] == pytest.approx(2.0 * (1 - 0.05), rel=1e-15)


def test_grad_norm_closed_form():
    n, c = T.grad_norm([np.array([3.0]), np.array([[0.0, 4.0]])], 1.0)
    assert n == 5.0 and c == pytest.approx(1.0 / (5.0 + 1e-6), rel=1e-15)
    assert T.grad_norm([np.zeros(3)], 1.0) == (0.0, 1.0)


def test_embed_grad_is_the_adjoint_of_the_lookup_and_its_difference_quotient():
    rng = np.random.default_rng(3)
    V, H, n, s = 7, 5, 30, 1.5
    ids = rng.integers(0, V, n)
    E, dy, D = rng.standard_normal((V, H)), rng.standard_normal((n, H)), rng.standard_normal((V, H))
    dE, mag, cnt = T.embed_grad(ids, dy, V, s)
    assert (dE * D).sum() == pytest.approx((dy * (s * D[ids])).sum(), rel=1e-12)
    loss = lambda t: (dy * (s * t[ids])).sum()  # noqa: E731
    assert (loss(E + 1e-3 * D) - loss(E - 1e-3 * D)) / 2e-3 == pytest.approx((dE * D).sum(), rel=1e-9)
    assert cnt.sum() == n and (mag >= np.abs(dE) - 1e-12).all()
    pad, _, _ = T.embed_grad(ids, dy, V, s, padding_id=int(ids[0]))
    assert not pad[ids[0]].any() and np.array_equal(np.delete(pad, ids[0], 0), np.delete(dE, ids[0], 0))


def test_embed_rows_rounds_once_and_zeroes_bad_ids():
    w = np.array([[1.0, 1 / 3], [2.0, -0.1]], np.float32)
    y = T.embed_rows(w, [1, -1, 2, 0], 0.1)
    assert np.array_equal(y[0], (w[1] * np.float32(0.1))) and not y[1].any() and not y[2].any()
    assert np.array_equal(y[3], w[0] * np.float32(0.1)) and math.isfinite(float(y.sum()))
