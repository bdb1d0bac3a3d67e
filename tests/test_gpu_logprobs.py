"""Log probabilities over logits (q4nx_token_logprobs) against float64.

Picks are on fp32 values on both sides: equal.  Sums: an exponential carries
2^-23 relative (one unit of the instruction) and the roundings of its exponent,
3 |d| 2^-24 with d = y - max; a value passes at most 160 additions in its lane, 12
in the wave's and rows' trees and, joined with other parts, the exponentials of
six levels and of up to four parts a lane, whose distances add up to its own.  So rest is off by at most
  r = 2^-23 (120 + 3 spread)  relative to 1 + rest,  spread = sum p |d|,
log1p and the final subtractions by 2^-23 each of their values:
  |logp - ref| <= r + 2^-22 (|d| + lz),   |H - ref| <= (r (1 + spread) + 2^-22 (lz + spread)) * 2.
For spread the weights are the probabilities; e |d| peaks at |d| = 1, so terms of
large |d| add little.  Where rest is small (a sharp row) r applies to rest alone.
fp32 ends at 2^-126: each of the n exponentials below it may count as 0 in rest
(2^-126 each), and in sum e |d| (|d| <= 126 ln 2 + 20 < 128 where e is above 2^-150
at all), which adds n 2^-126 to the first bound and n 2^-119 to the second.
"""
import math

import numpy as np
import pytest

import oracle
import synth

from _gpu import dev_f32, dev_i32, have_gpu, host, q, torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


def _run(y, n, tokens, k, ws=None, entropy=True):
    M, ldy = y.shape
    c = tokens.shape[1]
    print(f"logprobs M={M} n={n} ldy={ldy} tokens={c} k={k}", flush=True)
    out = {"logp": torch.full((M, c), -7.0, device="cuda") if c else None,
           "entropy": torch.full((M,), -7.0, device="cuda") if entropy else None,
           "top_ids": torch.full((M, k), -7, dtype=torch.int32, device="cuda") if k else None,
           "top_logp": torch.full((M, k), -7.0, device="cuda") if k else None}
    if ws is None:
        ws = torch.full((q().token_logprobs_ws(n, M, k),), 0xAB, dtype=torch.uint8, device="cuda")
    q().token_logprobs(dev_f32(y), n, M, ws, tokens=dev_i32(tokens) if c else None, n_tok=c, k=k, ldy=ldy, **out)
    return {name: None if v is None else host(v) for name, v in out.items()}


def _same_kind(got, want):
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    np.testing.assert_array_equal(got[inf], want[inf])
    return np.isfinite(want)


def _check(got, y, n, tokens, k, rows=None):
    for m in range(y.shape[0]) if rows is None else rows:
        lp, H, ids, top, spread = oracle.token_logprobs_ref(y[m, :n], tokens[m].tolist(), k)
        if k:
            np.testing.assert_array_equal(got["top_ids"][m], ids, err_msg=f"row {m}")
        alive = np.isfinite(H)
        lz = 0.0
        if alive:
            with np.errstate(invalid="ignore"):
                v = np.asarray(y[m, :n], dtype=np.float64)
            mx = np.nanmax(v)
            lz = -oracle.token_logprobs_ref(y[m, :n], [int(np.nanargmax(v))], 0)[0][0]
            rest = math.expm1(lz)
            r = 2.0 ** -23 * (120 + 3 * spread) * min(1.0, rest) + n * 2.0 ** -126
        for g, w in ((got["logp"], lp), (got["top_logp"], top)):
            if g is None:
                continue
            g, w = g[m].astype(np.float64), np.asarray(w, dtype=np.float64)
            fine = _same_kind(g, w)
            if alive:
                tol = r + 2.0 ** -22 * (np.abs(w + lz) + lz)
                assert (np.abs(g - w)[fine] <= tol[fine]).all(), (m, g, w, tol)
        if got["entropy"] is not None:
            e = got["entropy"][m]
            assert np.isnan(e) == np.isnan(H)
            if alive:
                assert abs(e - H) <= 2 * (r * (1 + spread) + 2.0 ** -22 * (lz + spread)) + n * 2.0 ** -119, (m, e, H)


def _logits(tag, M, ldy, std=2.0):
    g = synth.rng("gpu-logprobs", tag, M, ldy)
    y = (std * g.standard_normal((M, ldy))).astype(np.float32)
    y[np.arange(M), g.integers(0, max(1, ldy // 2), M)] += 9
    return g, y


@pytest.mark.parametrize("n", [1, 2, 3, 31, 64, 255, 256, 257, 1000, 1023, 1024, 1025, 4095, 4096, 4097, 5001, 20000])
@pytest.mark.parametrize("k", [0, 1, 5, 20, 32])
def test_lengths(n, k):
    k = min(k, n)
    M, c = 3, 2
    g, y = _logits("len", M, n + (n % 3))
    tokens = g.integers(0, n, (M, c)).astype(np.int32)
    _check(_run(y, n, tokens, k), y, n, tokens, k)


@pytest.mark.parametrize("M,n", [(1, 151936), (2, 262144), (2, 262145), (1, 1 << 20), (40, 151936)])
def test_long_rows(M, n):
    """Both sizes of part, up to the most parts that a row can have."""
    g, y = _logits("long", M, n)
    tokens = g.integers(0, n, (M, 1)).astype(np.int32)
    _check(_run(y, n, tokens, 20), y, n, tokens, 20, rows=range(min(M, 2)))


def test_many_rows():
    M, n = 3001, 1500
    g, y = _logits("rows", M, n + 1)
    tokens = g.integers(0, n, (M, 1)).astype(np.int32)
    got = _run(y, n, tokens, 3)
    _check(got, y, n, tokens, 3, rows=list(range(40)) + list(range(M - 40, M)))
    z = y[:, :n].astype(np.float64)
    lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
    assert np.abs(got["logp"][:, 0] - (z[np.arange(M), tokens[:, 0]] - lse)).max() < 2.0 ** -22 * 200
    np.testing.assert_array_equal(got["top_ids"], np.argsort(-y[:, :n], axis=1, kind="stable")[:, :3])


@pytest.mark.parametrize("n", [700, 4500, 70000])
@pytest.mark.parametrize("M", [9, 600])
def test_masks(n, M):
    """Ruled-out tokens as -inf, as the type's lowest value and as NaN; rows that leave nothing, or one
    token, or fewer than k; runs of equal logits."""
    low = np.finfo(np.float32).min
    k, ldy = 20, n + 5
    g, y = _logits("mask", M, ldy)
    y[0] = -np.inf                                   # nothing left
    y[1] = np.nan
    y[2, :n] = -np.inf
    y[2, n - 1] = -3.0                               # one
    y[3, :] = np.where(g.random(ldy) < 0.995, -np.inf, y[3])
    y[4, :] = np.where(g.random(ldy) < 0.995, low, y[4])
    y[5, :] = np.where(g.random(ldy) < 0.3, np.nan, y[5])
    y[6, :] = low                                    # every token alike, at the lowest value
    y[7, :] = np.round(y[7])                         # many ties
    y[8, :n] = -np.inf
    y[8, 100:140] = y[8, 640:650] = 1.5              # two runs of equal logits
    y[:, n:] = 100.0                                 # past n: not a logit
    tokens = np.stack([g.integers(0, n, M), np.full(M, n - 1), np.full(M, -1), np.full(M, n), np.full(M, 2 ** 31 - 1)],
                      1).astype(np.int32)
    _check(_run(y, n, tokens, k), y, n, tokens, k, rows=range(9))


@pytest.mark.parametrize("n", [300, 6000])
def test_infinities_and_ranges(n):
    M = 6
    g, y = _logits("inf", M, n)
    y[0, [7, n - 2]] = np.inf                        # share the whole
    y[0, 8] = -np.inf
    y[1] = 0.0
    y[1, ::2] = -0.0                                 # zeros of either sign are equal
    y[2] *= np.float32(1e36)
    y[3, 50] = 200.0                                 # all but certain
    y[4, 60] = 25.0                                  # rest lies below 2^-24 of the whole
    y[5] = -np.abs(y[5]) - 1e30
    tokens = np.tile(np.array([7, 8, 50, 60], dtype=np.int32), (M, 1))
    _check(_run(y, n, tokens, 10), y, n, tokens, 10)


@pytest.mark.parametrize("n", [4096, 16384])
def test_crowded_lanes(n):
    """Many large values in few of a wave's lanes, more than the gathering space holds, with and without
    ties: the values lane l sees are those at 4 l .. 4 l + 3 of every 256."""
    M, k = 4, 32
    g, y = _logits("crowd", M, n, std=1.0)
    at = np.arange(n)
    lanes = (at // 4) % 64 < 31
    y[0, lanes] += 50
    y[1, lanes] = 50.0
    y[2, lanes] = 50 + np.floor(3 * g.random(lanes.sum()))
    y[3, lanes] = np.inf
    tokens = np.zeros((M, 1), np.int32)
    for rows in (1, M):     # the small and the large part, at 4096 and up
        big = np.tile(y, (1 if rows == 1 else 400, 1))
        t = np.zeros((len(big), 1), np.int32)
        got = _run(big, n, t, k)
        _check(got, big, n, t, k, rows=range(M))
        np.testing.assert_array_equal(got["top_ids"][-M:], got["top_ids"][:M])
    assert tokens.size == M


def test_parts_asked_for():
    """Any of the outputs may be left out, and given tokens may be as many as 64."""
    M, n = 3, 5000
    g, y = _logits("parts", M, n)
    tokens = g.integers(0, n, (M, 64)).astype(np.int32)
    none = np.zeros((M, 0), np.int32)
    _check(_run(y, n, tokens, 0, entropy=False), y, n, tokens, 0)
    _check(_run(y, n, none, 0), y, n, none, 0)
    _check(_run(y, n, none, 7, entropy=False), y, n, none, 7)
    dy, ids = dev_f32(y), torch.empty((M, 7), dtype=torch.int32, device="cuda")
    ws = torch.empty(q().token_logprobs_ws(n, M, 7), dtype=torch.uint8, device="cuda")
    q().token_logprobs(dy, n, M, ws, k=7, top_ids=ids)
    np.testing.assert_array_equal(host(ids), np.argsort(-y, axis=1, kind="stable")[:, :7])


def test_rows_at_any_element_and_stale_workspace():
    M, n = 5, 4099
    g, y = _logits("shift", M, n + 2)
    tokens = g.integers(0, n, (M, 1)).astype(np.int32)
    buf = torch.zeros(y.size + 1, device="cuda")
    buf[1:].copy_(dev_f32(y).reshape(-1))
    size = q().token_logprobs_ws(n, M, 4)
    ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    lp, ids = torch.empty((M, 1), device="cuda"), torch.empty((M, 4), dtype=torch.int32, device="cuda")
    q().token_logprobs(buf[1:], n, M, ws, tokens=dev_i32(tokens), n_tok=1, logp=lp, k=4, top_ids=ids, ldy=n + 2,
                       ws_bytes=size)
    _check({"logp": host(lp), "entropy": None, "top_ids": host(ids), "top_logp": None}, y, n, tokens, 4)
    assert (host(ws[size:]) == 0x5A).all()


@pytest.mark.parametrize("M,n", [(1, 30000), (300, 20000)])
def test_captured_replayed_and_on_another_stream(M, n):
    g, y = _logits("graph", M, n)
    tokens, k = g.integers(0, n, (M, 1)).astype(np.int32), 6
    dy, dt = dev_f32(y), dev_i32(tokens)
    lp, H = torch.empty((M, 1), device="cuda"), torch.empty(M, device="cuda")
    ids, top = torch.empty((M, k), dtype=torch.int32, device="cuda"), torch.empty((M, k), device="cuda")
    ws = torch.full((q().token_logprobs_ws(n, M, k),), 0xAB, dtype=torch.uint8, device="cuda")
    args = dict(tokens=dt, n_tok=1, logp=lp, entropy=H, k=k, top_ids=ids, top_logp=top)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q().token_logprobs(dy, n, M, ws, stream=s, **args)
    s.synchronize()
    eager = [host(t).copy() for t in (lp, H, ids, top)]
    _check(dict(zip(("logp", "entropy", "top_ids", "top_logp"), eager)), y, n, tokens, k, rows=range(min(M, 3)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q().token_logprobs(dy, n, M, ws, **args)
    for i in range(3):
        for t in (lp, H, ids, top):
            t.zero_()
        ws.fill_(i)
        graph.replay()
        for t, e in zip((lp, H, ids, top), eager):
            np.testing.assert_array_equal(host(t), e)


def test_same_bits_every_time():
    M, n = 64, 40000
    g, y = _logits("bits", M, n)
    tokens = g.integers(0, n, (M, 1)).astype(np.int32)
    a, b = _run(y, n, tokens, 20), _run(y, n, tokens, 20)
    for name in a:
        np.testing.assert_array_equal(a[name], b[name])


@pytest.mark.parametrize("k", [1, 7, 32])
def test_waves_that_take_many_chunks(k):
    """Enough rows that a wave streams several chunks of its row: rising, falling, level, masked at the
    start, and runs whose values keep passing the k-th so far."""
    M, n = 3000, 20001
    g = np.random.default_rng(11)
    y = (2 * g.standard_normal((8, n))).astype(np.float32)
    y[0].sort()
    y[1] = np.sort(y[1])[::-1]
    y[2] = 1.25
    y[3, :9000] = -np.inf
    y[4, ::2] = np.arange(0, n, 2) / 1000
    y[5] = np.floor(np.arange(n) / 300)
    y[6, :] = np.finfo(np.float32).min
    y[6, n - 5:] = 3
    big = np.tile(y, (M // 8, 1))
    tokens = np.full((M, 1), n - 2, np.int32)
    got = _run(big, n, tokens, k)
    _check(got, big, n, tokens, k, rows=range(8))
    for name in ("logp", "entropy", "top_ids", "top_logp"):
        np.testing.assert_array_equal(got[name].reshape(M // 8, 8, -1), np.broadcast_to(got[name][:8].reshape(1, 8, -1), (M // 8, 8, got[name][0].size)))


def _run_many(rows, M, n, tokens, k):
    """A call over M rows that repeat the given ones (laid out on the device), with stale outputs; and the
    least chunks of 2048 logits that some wave took, from the records of parts that a call without
    alternatives leaves in its workspace: 16 bytes a part, the last 4 of them 0."""
    y = dev_f32(rows).repeat(M // len(rows), 1)
    print(f"logprobs M={M} n={n} k={k}", flush=True)
    out = {"logp": torch.full((M, 1), -7.0, device="cuda"), "entropy": torch.full((M,), -7.0, device="cuda"),
           "top_ids": torch.full((M, k), -7, dtype=torch.int32, device="cuda"), "top_logp": torch.full((M, k), -7.0, device="cuda")}
    dt = torch.from_numpy(tokens).cuda().repeat(M // len(rows), 1)
    size = q().token_logprobs_ws(n, M, k)
    ws = torch.full((size + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    q().token_logprobs(y, n, M, ws, tokens=dt, n_tok=1, k=k, ws_bytes=size, **out)
    assert bool((ws[size:] == 0xAB).all())
    got = {name: v.reshape(M // len(rows), len(rows), -1) for name, v in out.items()}
    for name, v in got.items():     # the same row, the same bits, wherever it lies
        v = v.view(torch.int32)
        assert bool((v == v[:1]).all()), name
    got = {name: host(v[0]) for name, v in got.items()}
    got["entropy"] = got["entropy"][:, 0]
    ws.fill_(0xAB)
    q().token_logprobs(y, n, M, ws, entropy=out["entropy"], ws_bytes=q().token_logprobs_ws(n, M, 0))
    parts = int((host(ws)[:size // 16 * 16].view(np.int32).reshape(-1, 4)[:, 3] == 0).sum()) // M
    return got, math.ceil(n / parts / 2048)


@pytest.mark.parametrize("n,M", [(65536, 16384), (151936, 16384), (151936, 4096)])
def test_level_rows_in_a_large_batch(n, M):
    """Rows whose many logits are alike, so that every addition of a long sum errs the same way, and rows
    whose maximum rises slowly all along, in batches so large that a wave takes many chunks: the error's
    bound does not grow with the batch."""
    g = np.random.default_rng(n)
    y = np.empty((8, n), np.float32)
    for i, d in enumerate((-0.76, -2.8, -2.05, -0.58, -5.3)):
        y[i] = d
        y[i, 7 * i] = 0.0
    y[5] = np.arange(n, dtype=np.float32) * np.float32(1e-4)
    y[6] = np.arange(n, dtype=np.float32) * np.float32(1e-6)
    y[7] = -1.37 + 1e-3 * g.standard_normal(n)
    tokens = np.full((8, 1), n - 3, np.int32)
    got, chunks = _run_many(y, M, n, tokens, 2)
    assert chunks >= 4
    _check(got, y, n, tokens, 2)


@pytest.mark.parametrize("k", [1, 20, 32])
@pytest.mark.parametrize("n,M", [(20001, 8192), (30001, 16384)])
def test_waves_that_take_five_chunks_and_more(n, M, k):
    """A threshold carried over many chunks, a gathering space that fills up and is cut down again and
    again, a maximum that rises many times, and a first bound only after chunks that are masked whole."""
    g = np.random.default_rng(n + k)
    y = (2 * g.standard_normal((16, n))).astype(np.float32)
    y[1].sort()
    y[2] = np.sort(y[2])[::-1]
    y[3] = 1.25
    y[4, :9000] = -np.inf
    y[5, ::2] = np.arange(0, n, 2) / 1000
    y[6] = np.floor(np.arange(n) / 300)
    y[7, :] = np.finfo(np.float32).min
    y[7, n - 5:] = 3
    y[8] = np.round(2 * y[8]) / 2                        # ties everywhere
    y[9] = y[9] / 4 + np.arange(n) / 4000                # more above the threshold in every chunk
    y[10, :n - 3000] = np.nan
    y[11] = np.where(g.random(n) < 0.999, -np.inf, y[11])   # fewer than k a chunk, for several chunks
    y[12] = np.repeat(np.arange(n // 100 + 1), 100)[:n] % 37
    y[13, :] = -np.inf
    y[13, n - 7] = y[13, 5] = -4.0
    y[14, 2048 * 3:] += 60                               # one rise, late
    y[15, ::1024] = np.inf
    tokens = g.integers(0, n, (16, 1)).astype(np.int32)
    tokens[:3, 0] = n - 1
    got, chunks = _run_many(y, M, n, tokens, k)
    assert chunks >= 5
    _check(got, y, n, tokens, k)
