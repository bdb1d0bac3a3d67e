"""Residual addition and RMS norm (q4nx_add_rmsnorm) against float64.

r_out is one fp32 addition: equal bit for bit to numpy's.  x: the sum of D
squares is off by at most D + 8 roundings of 2^-24 relative, of which the root
halves the effect, four more roundings follow, and the rounding to bf16 is half
a step, 2^-8 relative (or half the least subnormal):
  |x - x_ref| <= (2^-8 + (D / 2 + 16) 2^-24 (1 + 2^-8)) |x_ref| + 2^-134.
s itself carries one fp32 rounding, so the reference takes the rounded sum.
"""
import numpy as np
import pytest

import oracle
import synth

from _gpu import dev_bf16, dev_f32, have_gpu, host, q, torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

EPS = 1e-6


def _check_x(x_bits, s32, w_bits, eps):
    _, want = oracle.add_rmsnorm_ref(None, s32, synth.bf16_to_f32(w_bits), eps)
    D = s32.shape[1]
    got = synth.bf16_to_f32(x_bits.view(np.uint16)).astype(np.float64)
    tol = (2.0 ** -8 + (D / 2 + 16) * 2.0 ** -24 * (1 + 2.0 ** -8)) * np.abs(want) + 2.0 ** -134
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def _inputs(M, D, tag="norm"):
    g = synth.rng("gpu-norm", tag, M, D)
    y = g.standard_normal((M, D), dtype=np.float32)
    r = 5 * g.standard_normal((M, D), dtype=np.float32)
    r[:, :: max(1, D // 3)] *= 40
    w = synth.bf16_bits(1 + 0.3 * g.standard_normal(D))
    return y, r, w


SIZES = [(1, 1), (3, 2), (2, 3), (5, 63), (4, 64), (9, 80), (7, 127), (2048, 128), (3, 255), (3, 256), (3, 257), (5, 511),
         (4, 512), (3, 513), (2, 1023), (2, 1024), (2, 1026), (3, 2048), (2, 2049), (1, 2560), (65, 2560),
         (3, 4095), (33, 4096), (2, 4097), (1, 8192), (2, 8193), (2, 12289), (1, 16384), (2, 16385), (1, 28672),
         (2, 32767), (2, 32768)]


@pytest.mark.parametrize("M,D", SIZES)
def test_residual_and_norm(M, D):
    print(f"norm {M} x {D}", flush=True)
    y, r, w = _inputs(M, D)
    x = torch.full((M * D + 8,), -1, dtype=torch.int16, device="cuda")
    r_out = torch.full((M * D + 8,), -7.0, device="cuda")
    q().add_rmsnorm(dev_f32(r), dev_bf16(w), M, D, EPS, x, y=dev_f32(y), r_out=r_out)
    s = y + r
    np.testing.assert_array_equal(host(r_out)[:M * D].reshape(M, D), s)
    _check_x(host(x)[:M * D].reshape(M, D), s, w, EPS)
    assert (host(x)[M * D:] == -1).all() and (host(r_out)[M * D:] == -7.0).all()


@pytest.mark.parametrize("M,D", [(2, 128), (3, 100), (2, 2560), (2, 4097), (1, 9000)])
@pytest.mark.parametrize("where", ["r", "y", "none", "norm only"])
def test_in_place_and_without_outputs(M, D, where):
    y, r, w = _inputs(M, D, "place")
    dy, dr, x = dev_f32(y), dev_f32(r), torch.empty((M, D), dtype=torch.int16, device="cuda")
    r_out = {"r": dr, "y": dy}.get(where)
    q().add_rmsnorm(dr, dev_bf16(w), M, D, EPS, x, y=None if where == "norm only" else dy, r_out=r_out)
    s = r if where == "norm only" else y + r
    _check_x(host(x), s, w, EPS)
    np.testing.assert_array_equal(host(dr), s if where == "r" else r)
    np.testing.assert_array_equal(host(dy), s if where == "y" else y)


@pytest.mark.parametrize("D", [128, 513, 2560])
def test_arrays_at_any_element(D):
    """Every array one element off its allocation's alignment."""
    M = 3
    y, r, w = _inputs(M, D, "shift")

    def shifted(t):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:].copy_(t.reshape(-1))
        return buf[1:]
    x, r_out = torch.zeros(M * D + 1, dtype=torch.int16, device="cuda")[1:], torch.zeros(M * D + 1, device="cuda")[1:]
    q().add_rmsnorm(shifted(dev_f32(r)), shifted(dev_bf16(w)), M, D, EPS, x, y=shifted(dev_f32(y)), r_out=r_out)
    np.testing.assert_array_equal(host(r_out).reshape(M, D), y + r)
    _check_x(host(x).reshape(M, D), y + r, w, EPS)


def test_rows_out_of_the_ordinary():
    M, D = 6, 300
    y, r, w = _inputs(M, D, "odd")
    y[:] = 0
    r[0] = 0                                  # eps alone under the root
    r[1] *= np.float32(1e-25)                 # squares underflow: eps decides
    r[2] *= np.float32(1e15)
    r[3, 5] = np.inf
    r[4, 7] = np.nan
    x = torch.empty((M, D), dtype=torch.int16, device="cuda")
    q().add_rmsnorm(dev_f32(r), dev_bf16(w), M, D, EPS, x, y=dev_f32(y))
    got = host(x)
    _check_x(got[[0, 1, 2, 5]], r[[0, 1, 2, 5]], w, EPS)
    v = synth.bf16_to_f32(got.view(np.uint16))
    assert (v[0] == 0).all() and np.isnan(v[4]).all()
    assert np.isnan(v[3, 5]) and (np.delete(v[3], 5) == 0).all()
    # no eps: a row of zeros has no direction
    q().add_rmsnorm(dev_f32(r[:1]), dev_bf16(w), 1, D, 0.0, x)
    assert np.isnan(synth.bf16_to_f32(host(x)[0].view(np.uint16))).all()


def test_captured_replayed_and_on_another_stream():
    M, D = 5, 2560
    y, r, w = _inputs(M, D, "graph")
    dy, dr, dw = dev_f32(y), dev_f32(r), dev_bf16(w)
    x, r_out = torch.empty((M, D), dtype=torch.int16, device="cuda"), torch.empty((M, D), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q().add_rmsnorm(dr, dw, M, D, EPS, x, y=dy, r_out=r_out, stream=s)
    s.synchronize()
    eager = host(x)
    _check_x(eager, y + r, w, EPS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q().add_rmsnorm(dr, dw, M, D, EPS, x, y=dy, r_out=r_out)
    for _ in range(3):
        x.zero_()
        r_out.zero_()
        graph.replay()
        np.testing.assert_array_equal(host(x), eager)
        np.testing.assert_array_equal(host(r_out), y + r)


def test_many_rows():
    """More rows than a grid dimension of 65535 would hold."""
    M, D = 70000, 8
    y, r, w = _inputs(M, D, "many")
    x = torch.empty((M, D), dtype=torch.int16, device="cuda")
    q().add_rmsnorm(dev_f32(r), dev_bf16(w), M, D, EPS, x, y=dev_f32(y))
    _check_x(host(x), y + r, w, EPS)


@pytest.mark.parametrize("D", [4, 100, 256, 300, 700, 1025, 2560, 4097, 9000, 20000])
@pytest.mark.parametrize("place", ["apart", "in place", "norm only"])
def test_rows_whose_squares_leave_fp32(D, place):
    """Finite rows whose squares overflow or vanish in fp32 keep their x, beside rows that do neither, an
    infinity and a NaN.  Without eps, with one that counts beside the smallest squares, and with the usual
    one.  The bound is the file's: the rows are scaled by powers of two, and an element that this takes
    below 2^-126 has |x| < 2^-134 here (|w| < 4, and x is at most sqrt(D) of s over the row's largest)."""
    scales = [1.0, 2e19, 1e25, 3e37, 1e-20, 1e-25, 1e-37, 1e-40, 1.0, 1.0]
    M = len(scales)
    _, r, w = _inputs(M, D, "range")
    r = (r / np.abs(r).max(axis=1, keepdims=True) * np.array(scales)[:, None]).astype(np.float32)
    r[2, 1] = 1e-25                               # far below its row
    r[8, 0], r[9, 2] = np.inf, np.nan
    y = np.zeros_like(r) if place == "norm only" else (r / 4).astype(np.float32)
    s = y + r
    for eps in (0.0, 1e-44, 1e-30, EPS):
        dr, x = dev_f32(r), torch.full((M, D), -1, dtype=torch.int16, device="cuda")
        q().add_rmsnorm(dr, dev_bf16(w), M, D, eps, x, y=None if place == "norm only" else dev_f32(y),
                        r_out=dr if place == "in place" else None)
        got = host(x)
        _check_x(got[:8], s[:8], w, float(np.float32(eps)))
        if place == "in place":
            np.testing.assert_array_equal(host(dr), s)
        v = synth.bf16_to_f32(got.view(np.uint16))
        assert np.isnan(v[8, 0]) and (v[8, 1:] == 0).all() and np.isnan(v[9]).all()


@pytest.mark.parametrize("D", [64, 600, 4096])
def test_rows_of_zeros_with_any_eps(D):
    """Zeros over the root of eps are zeros, however small eps is; the row beside them keeps its values."""
    r = np.zeros((3, D), np.float32)
    r[1] = np.linspace(-1e-24, 1e-24, D, dtype=np.float32)
    w = synth.bf16_bits(np.ones(D))
    for eps in (1e-6, 1e-30, 1e-38, 1e-45):
        x = torch.full((3, D), -1, dtype=torch.int16, device="cuda")
        q().add_rmsnorm(dev_f32(r), dev_bf16(w), 3, D, eps, x)
        _check_x(host(x), r, w, float(np.float32(eps)))
