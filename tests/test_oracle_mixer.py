"""Pins for the mixer half of the oracle: closed forms and library routines."""
import numpy as np
import pytest

import oracle


def test_rmsnorm_rows_have_unit_mean_square():
    rng = np.random.default_rng(0)
    x, r = rng.standard_normal((5, 24)), rng.standard_normal((5, 24))
    y, s = oracle.rmsnorm(x, np.ones(24), 0.0, r)
    np.testing.assert_allclose(np.mean(y * y, axis=1), 1.0, rtol=1e-13)
    np.testing.assert_allclose(s, x + r)
    y2, _ = oracle.rmsnorm(x, 3.0 * np.ones(24), 0.0, r)
    np.testing.assert_allclose(y2, 3.0 * y)


def test_quant_rows_reach_127_and_stay_within_half_a_step():
    rng = np.random.default_rng(1)
    t = rng.standard_normal((7, 40)).astype(np.float32)
    t[3] = 0.0
    q, step = oracle.quant_rows_q8(t)
    assert np.all(np.max(np.abs(q[[0, 1, 2, 4, 5, 6]].astype(int)), axis=1) == 127)
    assert not q[3].any() and step[3] == 0.0
    assert np.all(np.abs(q * step[:, None] - t) <= 0.5 * step[:, None] * (1 + 1e-5))


def test_rmsnorm_q8_stands_for_the_norm():
    rng = np.random.default_rng(2)
    x, r, w = rng.standard_normal((6, 64)), rng.standard_normal((6, 64)), 1 + 0.1 * rng.standard_normal(64)
    x, r, w = (a.astype(np.float32) for a in (x, r, w))
    q, scale, _ = oracle.rmsnorm_q8(x, w, 1e-6, r)
    y, _ = oracle.rmsnorm(x, w, 1e-6, r)
    assert np.all(np.abs(q * scale[:, None] - y) <= 0.5001 * scale[:, None])


def test_linear_i8_is_the_matrix_product():
    rng = np.random.default_rng(3)
    xq, wq = rng.integers(-127, 128, (5, 48)), rng.integers(-127, 128, (7, 48))
    y = oracle.linear_i8(xq, 0.5 * np.ones(5), wq, 2.0 * np.ones(7), np.arange(7.0))
    np.testing.assert_array_equal(y, xq.astype(float) @ wq.T.astype(float) + np.arange(7.0))


def test_gated_delta_closed_forms():
    rng = np.random.default_rng(4)
    T, dk, dv = 6, 8, 3
    k = np.eye(8)[:T, None, :]                     # orthonormal keys: nothing is taken out
    q, v = rng.standard_normal((T, 1, dk)), rng.standard_normal((T, 1, dv))
    one, zero, off = np.ones((T, 1)), np.zeros((T, 1)), np.array([0, T])
    o, S = oracle.gated_delta(q, k, v, zero, one, off, scale=1.0, unit_qk=False)
    np.testing.assert_allclose(S[0, 0, :T], v[:, 0], atol=1e-14)
    np.testing.assert_allclose(o[-1, 0], q[-1, 0, :T] @ v[:, 0], atol=1e-13)
    # beta = 0 without decay leaves the state; beta = 1 replaces what the key holds
    S0 = rng.standard_normal((1, 1, dk, dv))
    _, S = oracle.gated_delta(q, k, v, zero, zero, off, scale=1.0, unit_qk=False, state=S0)
    np.testing.assert_allclose(S, S0)
    _, S = oracle.gated_delta(q, k, v, zero, one, off, scale=1.0, unit_qk=False, state=S0)
    np.testing.assert_allclose(S[0, 0, :T], v[:, 0], atol=1e-13)
    # g = -inf forgets everything before the token
    g = zero.copy(); g[3] = -np.inf
    o, _ = oracle.gated_delta(q, k, v, g, one, off, scale=1.0, unit_qk=False, state=S0)
    o2, _ = oracle.gated_delta(q[3:], k[3:], v[3:], zero[3:], one[3:], np.array([0, 3]), scale=1.0, unit_qk=False)
    np.testing.assert_allclose(o[3:], o2, atol=1e-13)


def test_gated_delta_splits_and_head_groups():
    rng = np.random.default_rng(5)
    T, hk, hv, dk, dv = 9, 2, 6, 8, 4
    q, k = rng.standard_normal((2, T, hk, dk))
    v, g, b = rng.standard_normal((T, hv, dv)), -rng.random((T, hv)), rng.random((T, hv))
    o, S = oracle.gated_delta(q, k, v, g, b, np.array([0, T]), scale=0.3, unit_qk=True)
    o1, S1 = oracle.gated_delta(q[:4], k[:4], v[:4], g[:4], b[:4], np.array([0, 4]), scale=0.3, unit_qk=True)
    o2, S2 = oracle.gated_delta(q[4:], k[4:], v[4:], g[4:], b[4:], np.array([0, T - 4]), scale=0.3, unit_qk=True, state=S1)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o, atol=1e-13)
    np.testing.assert_allclose(S2, S, atol=1e-13)
    for h in range(hv):  # each value head alone, with key head h // 3
        oh, _ = oracle.gated_delta(q[:, h // 3:h // 3 + 1], k[:, h // 3:h // 3 + 1], v[:, h:h + 1], g[:, h:h + 1],
                                   b[:, h:h + 1], np.array([0, T]), scale=0.3, unit_qk=True)
        np.testing.assert_allclose(oh[:, 0], o[:, h], atol=1e-13)
