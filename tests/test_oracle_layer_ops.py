"""Pins of the float64 definitions of the operators around the recurrence."""
import numpy as np
import pytest

from oracle import layer_ops as L


def test_short_conv_of_an_impulse_is_the_reversed_taps():
    w = np.array([[1.0, 2.0, 3.0, 4.0]])
    x = np.zeros((6, 1))
    x[1] = 1.0
    y, _, _, last = L.short_conv(x, w, act=False)
    np.testing.assert_array_equal(y[:, 0], [0, 4, 3, 2, 1, 0])
    np.testing.assert_array_equal(last[:, 0], [0, 0, 0])


@pytest.mark.parametrize("cut", [0, 1, 2, 5, 9])
def test_short_conv_in_two_parts_is_the_whole(cut):
    r = np.random.default_rng(0)
    x, w, b, h = r.normal(size=(9, 5)), r.normal(size=(5, 4)), r.normal(size=5), r.normal(size=(3, 5))
    whole, _, _, end = L.short_conv(x, w, b, h)
    y0, _, _, mid = L.short_conv(x[:cut], w, b, h)
    y1, _, _, end2 = L.short_conv(x[cut:], w, b, mid)
    np.testing.assert_allclose(np.concatenate([y0, y1]), whole, rtol=1e-13)
    np.testing.assert_array_equal(end, end2)


def test_silu_limits():
    np.testing.assert_allclose(L.silu([0.0, 1e3, -1e3]), [0.0, 1e3, 0.0], atol=1e-300)
    np.testing.assert_allclose(L.silu(1.0), 1.0 / (1.0 + np.exp(-1.0)), rtol=1e-15)


def test_scan_of_no_tokens_keeps_the_state_and_terms_bound_the_output():
    r = np.random.default_rng(1)
    S0 = r.normal(size=(4, 3, 5))
    _, S, _, _ = L.scan(np.zeros((0, 4, 3)), np.zeros((0, 2, 5)), np.zeros((0, 2, 5)), np.zeros((0, 4)), -np.ones(4),
                        np.ones(4), S0)
    np.testing.assert_array_equal(S, S0)
    y, _, size, _ = L.scan(r.normal(size=(7, 4, 3)), r.normal(size=(7, 2, 5)), r.normal(size=(7, 2, 5)),
                           r.uniform(0, 1, (7, 4)), -np.ones(4), r.normal(size=4), S0)
    assert np.all(np.abs(y) <= size * (1 + 1e-12))


def test_gated_norm_closed_forms():
    z = np.full((1, 4), 50.0)                                  # silu(50) = 50 to 1e-20
    y = np.array([[3.0, 4.0, 1.0, 1.0]])
    out = L.gated_norm(y, z, np.ones(4), 2, 0.0, True)
    np.testing.assert_allclose(out, 50 * np.array([[3 / np.sqrt(12.5), 4 / np.sqrt(12.5), 1, 1]]), rtol=1e-13)
    np.testing.assert_allclose(L.gated_norm(y, z, np.array([2.0, 1.0]), 2, 0.0, False),
                               np.array([[6 / np.sqrt(12.5), 4 / np.sqrt(12.5), 2, 1]]), rtol=1e-13)


def test_accept_cases():
    p = np.array([[0.5, 0.5, 0.0], [0.2, 0.3, 0.5], [0.0, 0.0, 1.0]])
    q = np.array([[0.25, 0.75, 0.0], [0.6, 0.2, 0.2]])
    assert L.accept([0, 0], p, [0.9, 0.3, 0.0], q) == (2, 2)   # .9 .25 < .5, .3 .6 < .2
    assert L.accept([0, 0], p, [0.9, 0.4, 0.0], q) == (1, 1)   # refused: residual (0, .1, .3)
    assert L.accept([0, 0], p, [0.9, 0.4, 0.26], q) == (1, 2)
    assert L.accept([1, 0], p, [0.7, 0.0, 0.99], q) == (0, 0)  # residual (.25, 0, 0)
    assert L.accept([1, 0], p, [0.7, 0.0, 0.6], q, 0) == (0, 1)  # no drafts: p_0 itself
    assert L.accept([2, 0], p, [0.0, 0.0, 0.4]) == (0, 0)      # certain draft of probability 0; p without it
    assert L.accept([7, 0], p, [0.0, 0.0, 0.6], q)[0] == 0     # a token that does not exist
    z = np.zeros((2, 3))
    assert L.accept([1], z, [0.0, 0.5], q[:1]) == (0, -1)


def test_accept_follows_the_target_distribution():
    """Over many uniforms the first emitted token has the target's frequencies."""
    r = np.random.default_rng(2)
    p, q = np.array([[0.1, 0.6, 0.3], [1.0, 0.0, 0.0]]), np.array([[0.5, 0.2, 0.3]])
    n, seen = 20000, np.zeros(3)
    for _ in range(n):
        x = r.choice(3, p=q[0])
        a, t = L.accept([x], p, r.uniform(size=2), q)
        seen[x if a else t] += 1
    assert np.all(np.abs(seen / n - p[0]) < 4 * np.sqrt(p[0] * (1 - p[0]) / n))
