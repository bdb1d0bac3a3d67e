"""Pins of the oracle's references for the tail of a step (oracle/tail.py), by
values worked out by hand and by other routes to the same number."""
import math

import numpy as np

import oracle


def test_lora_by_hand():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [5.0, 5.0]])
    A = np.array([[[1.0, 1.0], [0.0, 2.0]], [[2.0, 0.0], [math.nan, 7.0]]])      # E = 2, R = 2, K = 2
    B = np.array([[[1.0, 0.0], [0.0, 1.0], [1.0, -1.0]], [[1.0, math.nan]] * 3])   # N = 3
    base = np.arange(9.0).reshape(3, 3)
    y, mag = oracle.lora_ref(x, A, B, np.array([0.5, 2.0]), [0, 1, -1], base, ranks=[2, 1])
    # row 0: A x = (3, 4), B u = (3, 4, -1); row 1 uses rank 1: u = 6, B u = 6; row 2 has none
    np.testing.assert_array_equal(y, base + np.array([[1.5, 2.0, -0.5], [12.0, 12.0, 12.0], [0, 0, 0]]))
    np.testing.assert_array_equal(mag, np.array([[1.5, 2.0, 3.5], [12.0, 12.0, 12.0], [0, 0, 0]]))


def test_norm_by_hand():
    s, x = oracle.add_rmsnorm_ref(np.array([[1.0, 2.0]]), np.array([[2.0, 2.0]]), np.array([1.0, 0.5]), 0.0)
    np.testing.assert_array_equal(s, [[3.0, 4.0]])
    np.testing.assert_allclose(x, [[3 / math.sqrt(12.5), 2 / math.sqrt(12.5)]], rtol=1e-15)
    s, x = oracle.add_rmsnorm_ref(None, np.zeros((1, 4)), np.ones(4), 1e-6)
    assert not x.any()


def test_logprobs_by_hand():
    third = math.log(1 / 3)
    lp, H, ids, top, _ = oracle.token_logprobs_ref([0.0, -math.inf, 0.0, math.nan, 0.0], [0, 1, 3, 5, -1], 4)
    np.testing.assert_allclose(lp[0], third, rtol=1e-15)
    assert lp[1] == lp[2] == -math.inf and math.isnan(lp[3]) and math.isnan(lp[4])
    np.testing.assert_allclose(H, -third, rtol=1e-15)
    assert ids == [0, 2, 4, -1] and math.isnan(top[3])
    np.testing.assert_allclose(top[:3], [third] * 3, rtol=1e-15)
    # nothing left; a share of the whole among +inf; the type's lowest value is a value
    lp, H, ids, top, _ = oracle.token_logprobs_ref([-math.inf, math.nan], [0], 2)
    assert math.isnan(lp[0]) and math.isnan(H) and ids == [-1, -1]
    lp, H, ids, top, _ = oracle.token_logprobs_ref([math.inf, 3.0, math.inf], [0, 1], 3)
    np.testing.assert_allclose([lp[0], H], [-math.log(2), math.log(2)], rtol=1e-15)
    assert lp[1] == -math.inf and ids == [0, 2, 1] and top[2] == -math.inf
    low = float(np.finfo(np.float32).min)
    lp, H, ids, top, _ = oracle.token_logprobs_ref([low, low], [1], 1)
    np.testing.assert_allclose([lp[0], H], [-math.log(2), math.log(2)], rtol=1e-15)


def test_logprobs_against_the_plain_sum():
    g = np.random.default_rng(5)
    y = (3 * g.standard_normal(500)).astype(np.float32)
    lp, H, ids, top, _ = oracle.token_logprobs_ref(y, list(range(500)), 500)
    p = np.exp(y.astype(np.float64))
    p /= p.sum()
    np.testing.assert_allclose(lp, np.log(p), rtol=1e-13)
    np.testing.assert_allclose(H, -(p * np.log(p)).sum(), rtol=1e-13)
    np.testing.assert_array_equal(ids, np.argsort(-y, kind="stable"))
    # a sharp distribution: 1 - p of the likely token is 2 exp(-30)
    lp, H, _, _, _ = oracle.token_logprobs_ref([30.0, 0.0, 0.0], [0], 0)
    np.testing.assert_allclose(lp[0], -2 * math.exp(-30), rtol=1e-12)
    np.testing.assert_allclose(H, 2 * math.exp(-30) * 31, rtol=1e-12)
