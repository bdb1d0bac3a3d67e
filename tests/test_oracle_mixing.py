"""The float64 references of the cache, attention and linear attention, by hand-worked values and by
formulas that they do not use."""
import numpy as np

import oracle


def test_cache_layout_places():
    P, H, T, D = 2, 3, 32, 64
    x = np.arange(P * H * T * D).reshape(P, H, T, D)
    k, v = oracle.pack_k(x).reshape(-1), oracle.pack_v(x).reshape(-1)
    for p, h, t, d in [(0, 0, 0, 0), (1, 2, 31, 63), (0, 1, 17, 9), (1, 0, 8, 40)]:
        page = (p * H + h) * T * D
        assert k[page + (((t // 16) * (D // 8) + d // 8) * 16 + t % 16) * 8 + d % 8] == x[p, h, t, d]
        assert v[page + ((t // 8) * D + d) * 8 + t % 8] == x[p, h, t, d]
    np.testing.assert_array_equal(oracle.unpack_k(oracle.pack_k(x)), x)
    np.testing.assert_array_equal(oracle.unpack_v(oracle.pack_v(x)), x)


def test_rope_is_a_complex_product():
    g = np.random.default_rng(3)
    x, pos, f = g.standard_normal((5, 2, 64)), np.array([0, 1, -7, 1000, 2 ** 30]), 10.0 ** -np.arange(16.0)
    z = np.exp(1j * np.outer(pos, f))[:, None, :]
    y, mag = oracle.rope_ref(x, pos, f, 32, True)
    w = (x[..., 0:32:2] + 1j * x[..., 1:32:2]) * z
    np.testing.assert_allclose(y[..., 0:32:2], w.real, atol=1e-7)
    np.testing.assert_allclose(y[..., 1:32:2], w.imag, atol=1e-7)
    assert (np.abs(y) <= mag + 1e-12).all()
    y, mag = oracle.rope_ref(x, pos, f, 32, False)
    w = (x[..., :16] + 1j * x[..., 16:32]) * z
    np.testing.assert_allclose(y[..., :16], w.real, atol=1e-7)
    np.testing.assert_allclose(y[..., 16:32], w.imag, atol=1e-7)
    np.testing.assert_array_equal(y[..., 32:], x[..., 32:])
    np.testing.assert_array_equal(y[0], x[0])           # position 0 turns nothing
    assert (np.abs(y) <= mag + 1e-12).all()


def test_attention_by_hand():
    q, k = np.array([1.0, 0.0]), np.array([[0.0, 5.0], [np.log(3.0), 1.0]])
    v = np.array([[4.0, 0.0], [0.0, 8.0]])
    out, lse, mag, _ = oracle.attention_ref(q, k, v, 1.0)   # weights 1/4 and 3/4
    np.testing.assert_allclose(out, [1.0, 6.0])
    np.testing.assert_allclose(lse, np.log(4.0))
    np.testing.assert_allclose(mag, [1.0, 6.0])
    out, lse, _, _ = oracle.attention_ref(q, k[:0], v[:0], 1.0)
    assert (out == 0).all() and lse == -np.inf
    out, lse, _, _ = oracle.attention_ref(np.array([1.0, 1.0]), np.array([[-np.inf, 0.0], [2.0, 0.0]]), v, 1.0)
    np.testing.assert_allclose(out, v[1])
    np.testing.assert_allclose(lse, 2.0)


def test_attention_batch_sees_what_it_should():
    """Values that name their token: equal scores give the mean of the tokens seen."""
    q, D = np.zeros((4, 2, 64)), 64
    own = lambda s, h: (np.zeros((3, D)), np.repeat(10.0 * (s + 1) + np.arange(3.0), D).reshape(3, D))  # noqa: E731
    prefix = lambda h: (np.zeros((2, D)), np.full((2, D), 100.0))  # noqa: E731
    out, lse, _, _ = oracle.attention_batch_ref(q, [0, 2, 2, 3], [3, 3, 1], own, prefix, 1.0, 2)
    np.testing.assert_allclose(out[0, 0, 0], (200 + 10 + 11) / 4)           # two rows, three tokens: two seen
    np.testing.assert_allclose(out[1, 1, 5], (200 + 10 + 11 + 12) / 5)
    np.testing.assert_allclose(out[2, 0, 0], (200 + 30) / 3)
    np.testing.assert_allclose(lse[2, 0], np.log(3))
    assert np.isnan(out[3]).all()                                           # no sequence's row


def test_linear_attention_is_a_weighted_sum():
    g = np.random.default_rng(5)
    T, dk, dv = 9, 4, 3
    q, k, v = g.standard_normal((T, dk)), g.standard_normal((T, dk)), g.standard_normal((T, dv))
    d, S0 = -g.random(T), g.standard_normal((dk, dv))
    out, S, mag, A = oracle.linear_attn_ref(q, k, v, d, 0.5, S0)
    C = np.cumsum(d)
    for t in range(T):
        want = np.exp(C[t]) * (q[t] @ S0) + sum(np.exp(C[t] - C[j]) * (q[t] @ k[j]) * v[j] for j in range(t + 1))
        np.testing.assert_allclose(out[t], 0.5 * want, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S, np.exp(C[-1]) * S0 + sum(np.exp(C[-1] - C[j]) * np.outer(k[j], v[j]) for j in range(T)),
                               rtol=1e-12)
    assert (np.abs(out) <= mag + 1e-12).all() and (np.abs(S) <= A + 1e-12).all()
    d[4] = -np.inf                                                          # forgets all, an infinite state too
    S0[0, 0] = np.inf
    with np.errstate(invalid="ignore"):
        out, S, _, _ = oracle.linear_attn_ref(q, k, v, d, 0.5, S0)
    np.testing.assert_allclose(out[4], 0.5 * (q[4] @ k[4]) * v[4])
    assert np.isfinite(S).all()
