"""Rotation and append to the paged cache (q4nx_kv_append) against float64.

bf16: a cosine and a sine are off by at most 2^-24 (rounded from fp64) and the turn adds two roundings, each
relative to |a| + |b|, so 4 * 2^-24 (|a| + |b|), and the rounding to bf16 is half a step, 2^-8 relative (or half
the least subnormal):  |x - x_ref| <= 2^-8 |x_ref| + 4 (1 + 2^-8) 2^-24 (|a| + |b|) + 2^-134.
INT8: formed in fp64; the scale is one rounding to fp32 of max / 127 (relative 2^-24, beside fp64's own errors
2^-40), and code * scale is off by at most half a scale (2^-40 of it beside); a code of magnitude 127 by as much
as the scale's rounding times 127 more.
"""
import numpy as np
import pytest

import oracle
import synth

from _gpu import dev_bf16, dev_f32, dev_i32, have_gpu, host, q, torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

FILL = {"bf16": 0x7FC1, "int8": 77}


class Cache:
    """A cache of pages that hold a pattern, with its logical view."""

    def __init__(self, kind, H, D, page, pages):
        self.kind, self.H, self.D, self.page, self.pages = kind, H, D, page, pages
        n = pages * H * page * D
        if kind == "bf16":
            self.k, self.v = (dev_bf16(np.full(n, FILL[kind], np.uint16)) for _ in range(2))
            self.ks = self.vs = None
        else:
            self.k, self.v = (torch.full((n,), FILL[kind], dtype=torch.int8, device="cuda") for _ in range(2))
            self.ks, self.vs = (torch.full((pages * H * page,), -3.0, device="cuda") for _ in range(2))
        self.c = q().kv_cache(H, D, page, pages, self.k, self.v, k_scale=self.ks, v_scale=self.vs)

    def logical(self):
        """(k, v) as raw elements [slot, head, dim], and the scales [slot, head]."""
        P, H, T, D = self.pages, self.H, self.page, self.D
        raw = np.uint16 if self.kind == "bf16" else np.int8
        k = oracle.unpack_k(host(self.k).view(raw).reshape(P, H, T // 16, D // 8, 16, 8))
        v = oracle.unpack_v(host(self.v).view(raw).reshape(P, H, T // 8, D, 8))
        k, v = (x.transpose(0, 2, 1, 3).reshape(P * T, H, D) for x in (k, v))
        if self.kind == "bf16":
            return k, v, None, None
        return k, v, *(host(s).reshape(P, H, T).transpose(0, 2, 1).reshape(P * T, H) for s in (self.ks, self.vs))


def _check(kind, got, scale, want, mag, turned=True):
    if kind == "bf16":
        x = synth.bf16_to_f32(got.view(np.uint16)).astype(np.float64)
        tol = 2.0 ** -8 * np.abs(want) + (4 * (1 + 2.0 ** -8) * 2.0 ** -24 * mag if turned else 0) + 2.0 ** -134
        bad = ~(np.abs(x - want) <= tol)
    else:
        s = scale.astype(np.float64)
        top = np.abs(want).max(-1) / 127
        assert (np.abs(s - top) <= (2.0 ** -24 + 2.0 ** -40) * top + 2.0 ** -150).all()
        x = got.astype(np.float64) * s[..., None]
        tol = (0.5 + 2.0 ** -40 + 127 * 2.0 ** -24) * s[..., None] + 2.0 ** -149
        bad = ~(np.abs(x - want) <= tol)
        assert (np.abs(got.astype(int)) <= 127).all()
    assert not bad.any(), (np.argwhere(bad)[:4], x[bad][:4], want[bad][:4])


def _rows(g, M, n, D, bf16):
    x = g.standard_normal((M, n, D)).astype(np.float32)
    x[:, :, :: 17] *= 9
    return (synth.bf16_to_f32(synth.bf16_bits(x)), synth.bf16_bits(x)) if bf16 else (x, None)


def _dev(x, bits, pad=0):
    """[M, n * D (+ pad)] on the device, as int16 bits or fp32."""
    M = x.shape[0]
    flat = (bits if bits is not None else x).reshape(M, -1)
    if pad:
        flat = np.concatenate([flat, np.zeros((M, pad), flat.dtype)], 1)
    t = dev_bf16(flat) if bits is not None else dev_f32(flat)
    return t[:, : flat.shape[1] - pad] if pad else t


def _run(kind, M, H, KH, D, page, rot, interleaved, q_bf16, v_bf16, pad=0, with_q=True, seed=0, pos=None, slots=None,
         flags=None, stream=None):
    g = synth.rng("kv-append", kind, M, H, KH, D, page, rot, interleaved, seed)
    pages = -(-M // page) + 2
    if slots is None:
        slots = g.permutation(pages * page)[:M].astype(np.int32)
        if M > 3:
            slots[M // 2] = -1
    if pos is None:
        pos = g.integers(0, 1 << 20, M).astype(np.int32)
    f = (1e4 ** (-np.arange(rot // 2) * 2 / max(rot, 1))).astype(np.float32)
    xq, bq = _rows(g, M, H, D, q_bf16)
    xk, bk = _rows(g, M, KH, D, q_bf16)
    xv, bv = _rows(g, M, KH, D, v_bf16)
    cache = Cache(kind, KH, D, page, pages)
    q_out = torch.full((M * H * D + 8,), 0x7FC1, dtype=torch.int16, device="cuda")
    rope = q().rope(dev_f32(f), dev_i32(pos), rot, interleaved) if rot else None
    q().kv_append(cache.c, _dev(xk, bk, pad), _dev(xv, bv, pad), dev_i32(slots), M, rope=rope,
                  q=_dev(xq, bq, pad) if with_q else None, q_heads=H if with_q else None,
                  q_out=q_out[: M * H * D] if with_q else None, flags=flags, stream=stream)
    out = host(q_out)
    assert (out[M * H * D:] == 0x7FC1).all()
    if with_q:
        want, mag = oracle.rope_ref(xq, pos, f, rot, interleaved)
        _check("bf16", out[: M * H * D].reshape(M, H, D), None, want, mag, rot > 0)
    else:
        assert (out == 0x7FC1).all()
    k, v, ks, vs = cache.logical()
    # of rows with one slot the last counts
    last = {int(s): m for m, s in enumerate(slots) if 0 <= s < pages * page}
    at, rows = np.array(list(last), int), np.array(list(last.values()), int)
    want, mag = oracle.rope_ref(xk, pos, f, rot, interleaved)
    if len(at):
        _check(kind, k[at], ks[at] if ks is not None else None, want[rows], mag[rows], rot > 0)
        _check(kind, v[at], vs[at] if vs is not None else None, xv[rows].astype(np.float64), None, False)
    rest = np.setdiff1d(np.arange(pages * page), at)
    assert (k[rest] == FILL[kind]).all() and (v[rest] == FILL[kind]).all()
    if ks is not None:
        assert (ks[rest] == -3.0).all() and (vs[rest] == -3.0).all()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("M,H,KH,D,page,rot,interleaved,q_bf16,v_bf16,pad", [
    (1, 32, 8, 128, 64, 128, False, False, False, 0),
    (1, 1, 1, 64, 16, 16, True, True, True, 0),
    (2, 5, 5, 64, 16, 64, False, False, True, 3),
    (7, 14, 2, 128, 32, 64, False, True, False, 1),
    (17, 6, 3, 256, 16, 256, True, False, False, 0),
    (64, 16, 2, 256, 256, 128, True, True, False, 0),
    (65, 8, 8, 64, 1024, 32, False, True, True, 5),
    (300, 4, 1, 128, 16, 128, False, False, False, 7),
    (1025, 2, 2, 64, 64, 48, True, True, False, 0),
    (4100, 2, 1, 128, 128, 128, False, False, False, 0),
    (9, 4, 2, 128, 64, 0, False, False, False, 0),
])
def test_append(kind, M, H, KH, D, page, rot, interleaved, q_bf16, v_bf16, pad):
    print(f"append {kind} {M} {H}/{KH} x {D} page {page} rope {rot}", flush=True)
    _run(kind, M, H, KH, D, page, rot, interleaved, q_bf16, v_bf16, pad)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("first", [0, 1, 7, 8, 13])
@pytest.mark.parametrize("M", [1, 8, 40, 777, 4097])
def test_runs_of_neighbouring_slots(kind, first, M):
    """A prompt's tokens, from any place in a page."""
    slots = (first + np.arange(M)).astype(np.int32)
    pos = (70000 + np.arange(M)).astype(np.int32)
    _run(kind, M, 4, 2, 64, 16, 64, False, True, False, slots=slots, pos=pos)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_several_prompts_in_one_call(kind):
    """Runs that begin anywhere, one after the other, with padding between and behind."""
    slots = np.concatenate([np.arange(5, 38), [-1, -1], np.arange(96, 113), np.arange(50, 64), [-1] * 9, np.arange(80, 81)])
    _run(kind, len(slots), 2, 2, 128, 16, 128, False, False, False, slots=slots.astype(np.int32))


def test_without_q():
    _run("bf16", 19, 4, 2, 128, 16, 64, False, False, False, with_q=False)
    _run("int8", 19, 4, 2, 128, 16, 64, True, True, False, with_q=False)


def test_far_and_negative_positions():
    pos = np.array([0, 1, -1, 131071, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 999999937], np.int32)
    for kind in ("bf16", "int8"):
        _run(kind, 8, 2, 1, 128, 16, 128, False, False, False, pos=pos)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_the_same_slot_twice(kind):
    """The last of the rows with a slot is stored, wherever the others are."""
    g = synth.rng("kv-append-twice", kind)
    for M in (2, 9, 64, 1500, 5000):
        slots = g.integers(-1, max(2, M // 3), M).astype(np.int32)
        slots[0] = slots[-1] = 1
        _run(kind, M, 1, 1, 64, 16, 64, False, True, False, slots=slots, seed=M)


def test_slots_outside_the_cache():
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    _run("bf16", 6, 2, 1, 64, 16, 64, False, False, False, slots=np.array([-1, 3, -1, 7, 0, -1], np.int32), flags=flags)
    assert host(flags)[0] == 0
    slots = np.array([48, 3, -2, 2 ** 31 - 1, -2 ** 31, 47], np.int32)      # three pages of 16: 47 is the last
    for kind in ("bf16", "int8"):
        flags.zero_()
        _run(kind, 6, 2, 1, 64, 16, 64, False, False, False, slots=slots, flags=flags)
        assert host(flags)[0] == 1
        _run(kind, 6, 2, 1, 64, 16, 64, False, False, False, slots=slots)   # and without flags


def test_eight_bit_heads_out_of_the_ordinary():
    """Zeros, the least and largest numbers, and heads with an infinity or a NaN."""
    D, M = 64, 6
    x = np.zeros((M, 1, D), np.float32)
    x[1, 0, 3] = 1e-45
    x[2, 0] = np.linspace(-3e38, 3e38, D)
    x[3, 0, 5] = -np.inf
    x[4, 0, 6] = np.nan
    x[5, 0] = 1e-40 * np.arange(D)
    cache = Cache("int8", 1, D, 16, 1)
    q().kv_append(cache.c, _dev(x, None), _dev(x, None), dev_i32(np.arange(M)), M)
    for codes, scale in zip(cache.logical()[:2], cache.logical()[2:]):
        codes, scale = codes[:M, 0].astype(float), scale[:M, 0].astype(float)
        assert scale[0] == 0 and (codes[0] == 0).all()
        assert np.isinf(scale[3]) and (codes[3] == 0).all() and np.isnan(scale[4]) and (codes[4] == 0).all()
        for m in (1, 2, 5):     # a subnormal scale is off by half the least subnormal
            assert (np.abs(codes[m] * scale[m] - x[m, 0].astype(float)) <= (0.5 + 1e-4) * scale[m] + 127 * 2.0 ** -150).all()


def test_captured_and_on_another_stream():
    M, H, KH, D = 33, 4, 2, 128
    g = synth.rng("kv-append-graph")
    x = [dev_f32(g.standard_normal((M, n * D))) for n in (H, KH, KH)]
    pos, slots = dev_i32(np.arange(M) + 100), dev_i32(g.permutation(64)[:M])
    f = dev_f32(1e4 ** (-np.arange(64) / 64))
    caches = [Cache("int8", KH, D, 16, 4) for _ in range(2)]
    outs = [torch.zeros((M, H, D), dtype=torch.int16, device="cuda") for _ in range(2)]

    def call(i, stream=None):
        q().kv_append(caches[i].c, x[1], x[2], slots, M, rope=q().rope(f, pos, D), q=x[0], q_heads=H, q_out=outs[i], stream=stream)
    call(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(1)
    for shift in (0, 3, 11):
        pos += shift
        x[1].mul_(1.5)
        call(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        for a, b in zip(caches[0].logical(), caches[1].logical()):
            np.testing.assert_array_equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs[1].zero_()
    s.wait_stream(torch.cuda.current_stream())
    call(1, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("q_bf16,v_bf16", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("run", [True, False])
def test_rows_at_odd_strides(kind, q_bf16, v_bf16, run):
    """Rows that lie at no more than their element's alignment, in tiles of eight."""
    slots = (np.arange(777) + 3).astype(np.int32) if run else None
    _run(kind, 777, 3, 2, 128, 64, 64, False, q_bf16, v_bf16, pad=3, slots=slots)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("M,run", [(7, False), (700, False), (700, True)])
def test_eight_bit_codes_at_half_steps(D, M, run):
    """Codes are round(x / scale), half to even, at exact half steps and right beside them.

    Each row's largest value is 127 s for a whole s, which makes the scale s; the others are odd multiples of s / 2, and
    their neighbours in fp32 on either side: every code is known."""
    g = synth.rng("kv-append-half", D, M, run)
    s = g.integers(1, 1 << 14, M).astype(np.float64)
    s[0] = 49
    half = (2 * g.integers(0, 127, (M, 1, D)) + 1) * s[:, None, None] / 2 * g.choice([-1.0, 1.0], (M, 1, D))
    x = half.astype(np.float32)
    assert (x == half).all()
    side = g.integers(0, 4, x.shape)
    x = np.where(side == 0, np.nextafter(x, np.float32(0)), np.where(side == 1, np.nextafter(x, np.float32(np.inf) * np.sign(x)), x))
    x[0, 0, 1] = 73.5                                           # over 49: one and a half
    x[:, 0, 0] = 127 * s
    pages = M // 16 + 2
    slots = (np.arange(M) + 8 if run else g.permutation(pages * 16)[:M]).astype(np.int32)
    cache = Cache("int8", 1, D, 16, pages)
    q().kv_append(cache.c, _dev(x, None), _dev(x, None), dev_i32(slots), M)
    want = np.rint(x.astype(np.float64) / s[:, None, None])
    want[:, :, 1:] = np.clip(want[:, :, 1:], -127, 127)
    k, v, ks, vs = cache.logical()
    for codes, scale in ((k, ks), (v, vs)):
        np.testing.assert_array_equal(scale[slots, 0], s)
        bad = codes[slots] != want
        assert not bad.any(), (bad.sum(), x[bad][:4], codes[slots][bad][:4], want[bad][:4])
