"""Low-rank adapters beside a projection (q4nx_lora_add, q4nx_lora_add_batched)
against the float64 reference.

Tolerance: bf16 x bf16 products are exact in fp32, so an element of A x is off
by at most K roundings of 2^-23 (2^-24, doubled for a matrix core that truncates)
of sum |a x|.  Its three bf16 parts hold it exactly; scaling is one rounding, the
second product adds 3 R roundings, the parts of K 64 at most, the base two:
  |y - y_ref| <= 2^-23 ((K + 3 R + 80) sum |scale b| sum |a x| + |base| + |y_ref|).
"""
import numpy as np
import pytest

import oracle
import synth

from _gpu import dev_bf16, dev_f32, dev_i32, have_gpu, host, q, torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


class Case:
    """Inputs of one call and their device copies; adapters lie `pad` elements apart."""

    def __init__(self, tag, M, K, N, R, E, ids, ranks=None, pad=0, garbage=False):
        g = synth.rng("gpu-lora", tag, M, K, N, R, E)
        self.M, self.K, self.N, self.R, self.E = M, K, N, R, E
        self.x = synth.bf16_bits(g.standard_normal((M, K)))
        A = synth.bf16_bits(g.standard_normal((E, R, K)) / np.sqrt(K))
        B = synth.bf16_bits(g.standard_normal((E, N, R)) / np.sqrt(R))
        if garbage:      # what lies past an adapter's rank may hold anything
            for e in range(E):
                A[e, ranks[e]:] = 0x7FC0
                B[e, :, ranks[e]:] = 0x7F80
        self.A, self.B = synth.bf16_to_f32(A), synth.bf16_to_f32(B)
        self.scale = (0.25 + g.random(E)).astype(np.float32)
        self.ids = np.asarray(ids, dtype=np.int32)
        self.ranks = None if ranks is None else np.asarray(ranks, dtype=np.int32)
        self.base = g.standard_normal((M, N)).astype(np.float32)

        def arena(v):
            flat = np.full((E, v[0].size + pad), 0x7FC0, np.uint16)
            flat[:, :v[0].size] = v.reshape(E, -1)
            return dev_bf16(flat)
        self.dx, self.dids, self.dbase = dev_bf16(self.x), dev_i32(self.ids), dev_f32(self.base)
        self.table = q().lora_table(E, R, N, K, arena(A), arena(B), dev_f32(self.scale),
                                    ranks=None if ranks is None else dev_i32(self.ranks),
                                    a_stride=2 * (R * K + pad), b_stride=2 * (R * N + pad))

    def ref(self):
        return oracle.lora_ref(synth.bf16_to_f32(self.x), self.A, self.B, self.scale, self.ids, self.base, self.ranks)

    def check(self, y):
        want, mag = self.ref()
        tol = 2.0 ** -23 * ((self.K + 3 * self.R + 80) * mag + np.abs(self.base) + np.abs(want))
        assert np.isfinite(y).all()
        bad = np.abs(y - want) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(y - want).max())
        none = (self.ids < 0) | (self.ids >= self.E)
        np.testing.assert_array_equal(y[none], self.base[none])

    def run(self, in_place=False, ws=None):
        print(f"lora M={self.M} K={self.K} N={self.N} R={self.R} E={self.E} in_place={in_place}", flush=True)
        if ws is None:      # stale contents
            ws = torch.full((q().lora_ws(self.table, self.M),), 0xAB, dtype=torch.uint8, device="cuda")
        y = self.dbase.clone() if in_place else torch.full((self.M, self.N), float("nan"), device="cuda")
        q().lora_add(self.table, self.dx, self.dids, self.M, y, ws, base=None if in_place else self.dbase)
        out = host(y)
        self.flag = int(host(ws[:4].view(torch.int32))[0])
        return out


def _ids(kind, M, E, seed=1):
    g = np.random.default_rng(seed)
    return {"one": np.zeros(M), "each": np.arange(M) % E, "random": g.integers(0, E, M),
            "some": np.where(g.random(M) < 0.5, -1, g.integers(0, E, M)), "none": np.full(M, -1),
            "runs": np.sort(g.integers(0, E, M))[::-1]}[kind].astype(np.int32)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("M,kind", [(1, "one"), (1, "none"), (2, "each"), (8, "random"), (17, "one"), (16, "one"),
                                    (64, "each"), (64, "one"), (63, "some"), (33, "none")])
def test_decode_rows(M, kind, in_place):
    c = Case("decode", M, 512, 96, 16, 40, _ids(kind, M, 40))
    c.check(c.run(in_place))
    assert c.flag == 0


@pytest.mark.parametrize("M,kind,E", [(65, "one", 3), (128, "each", 128), (200, "random", 5), (255, "some", 9),
                                      (256, "runs", 4), (257, "runs", 4), (300, "each", 300), (400, "some", 7),
                                      (513, "one", 1), (1000, "runs", 6), (1024, "none", 2)])
def test_prompt_rows(M, kind, E):
    c = Case("prompt", M, 256, 64, 8, E, _ids(kind, M, E))
    c.check(c.run())
    c.check(c.run(in_place=True))
    assert c.flag == 0


@pytest.mark.parametrize("M", [3, 100, 300])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128, 200, 256])
def test_ranks_stored(R, M):
    c = Case("rank", M, 768, 160, R, 5, _ids("random", M, 5))
    c.check(c.run())


@pytest.mark.parametrize("M", [6, 90, 270])
def test_ranks_of_each_adapter(M):
    ranks = [0, 1, 7, 8, 9, 31, 33, 63, 64, 72]
    c = Case("mixed", M, 512, 64, 72, len(ranks), _ids("random", M, len(ranks)), ranks, garbage=True)
    c.check(c.run())
    c.ranks = np.array([-3, 1, 7, 8, 9, 31, 33, 63, 64, 1000], dtype=np.int32)     # clamped to 0..72
    c.A[~np.isfinite(c.A)] = 0
    c.B[~np.isfinite(c.B)] = 0
    d = Case("mixed", M, 512, 64, 72, len(ranks), c.ids, list(c.ranks))
    d.check(d.run())


@pytest.mark.parametrize("K,N", [(256, 32), (2560, 4096), (9728, 2560), (28672, 96), (256, 14336), (7424, 1056)])
@pytest.mark.parametrize("M", [1, 5, 70])
def test_shapes(M, K, N):
    c = Case("shape", M, K, N, 16, 3, _ids("random", M, 3))
    c.check(c.run())


@pytest.mark.parametrize("M", [4, 300])
def test_padded_arenas(M):
    c = Case("pad", M, 256, 64, 16, 3, _ids("random", M, 3), pad=24)
    c.check(c.run())


@pytest.mark.parametrize("M", [5, 64, 256, 270])
def test_ids_outside(M):
    ids = _ids("random", M, 4)
    ids[[0, 3]] = [4, -2]
    ids[2] = 2 ** 31 - 1
    ids[M - 1] = -2 ** 31
    c = Case("outside", M, 256, 64, 8, 4, ids)
    c.check(c.run())
    assert c.flag == 1
    ids[:] = -1
    c = Case("outside", M, 256, 64, 8, 4, ids)
    c.check(c.run())
    assert c.flag == 0


@pytest.mark.parametrize("M", [40, 200, 500])
def test_a_rows_bits_depend_on_its_own_inputs_only(M):
    c = Case("bits", M, 512, 128, 32, 6, _ids("random", M, 6))
    y0 = c.run()
    np.testing.assert_array_equal(c.run().view(np.int32), y0.view(np.int32))
    # the same rows in another order
    p = np.random.default_rng(3).permutation(M)
    c.dx, c.dids, c.dbase = dev_bf16(c.x[p]), dev_i32(c.ids[p]), dev_f32(c.base[p])
    np.testing.assert_array_equal(c.run().view(np.int32), y0[p].view(np.int32))
    # every row but 7 with another adapter
    ids = (c.ids + 1) % 6
    ids[7] = c.ids[7]
    c.dx, c.dids, c.dbase = dev_bf16(c.x), dev_i32(ids), dev_f32(c.base)
    np.testing.assert_array_equal(c.run()[7].view(np.int32), y0[7].view(np.int32))


def test_values_out_of_the_ordinary():
    """Infinities and NaN stay in their rows; large and small values keep their digits."""
    c = Case("inf", 6, 256, 64, 8, 2, [0, 1, 0, 1, 0, 0])
    c.x[1, 3] = 0x7F80                       # +inf
    c.x[2, 5] = 0x7FC0                       # NaN
    c.x[3] = synth.bf16_bits(synth.bf16_to_f32(c.x[3]) * np.float32(1e30))
    c.x[4] = synth.bf16_bits(synth.bf16_to_f32(c.x[4]) * np.float32(1e-30))
    c.base[4:5] = 0
    c.dx, c.dbase = dev_bf16(c.x), dev_f32(c.base)
    y = c.run()
    with np.errstate(invalid="ignore"):
        want, mag = c.ref()
    assert np.isnan(y[2]).all() and not np.isfinite(y[1]).any()
    for m in (0, 3, 4, 5):
        tol = 2.0 ** -23 * ((c.K + 3 * c.R + 80) * mag[m] + np.abs(c.base[m]) + np.abs(want[m]))
        assert (np.abs(y[m] - want[m]) <= tol).all(), m
    # an infinite A x against finite B: infinite of B's sign, as the formula has it
    c = Case("inf2", 1, 256, 32, 8, 1, [0], ranks=[1])
    c.x[:] = 0
    c.x[0, 0] = 0x7F80
    c.dx = dev_bf16(c.x)
    y = c.run()
    a0, b0 = c.A[0, 0, 0], c.B[0, :, 0]
    rest = c.A[0, 0, 1:]
    assert a0 != 0 and np.isfinite(rest).all() and (b0 != 0).all()
    np.testing.assert_array_equal(y[0], np.sign(b0) * np.sign(a0) * np.inf)


@pytest.mark.parametrize("M", [1, 9, 64, 300])
def test_batched_projections(M):
    """q, k and v of one layer, at different ranks: each job as its own call gives it, up to the
    order of its sums."""
    ids = _ids("some", M, 5)
    cs = [Case(f"qkv{i}", M, 512, n, r, 5, ids) for i, (n, r) in enumerate([(256, 16), (64, 40), (96, 128)])]
    for c in cs[1:]:
        c.x, c.dx = cs[0].x, cs[0].dx
    ys = [torch.full((M, c.N), float("nan"), device="cuda") for c in cs]
    jobs = q().lora_jobs([(c.table, c.dbase, y) for c, y in zip(cs, ys)])
    ws = torch.full((q().lora_batched_ws(jobs, M),), 0xCD, dtype=torch.uint8, device="cuda")
    print(f"lora batched M={M}", flush=True)
    q().lora_add_batched(jobs, cs[0].dx, cs[0].dids, M, ws)
    for c, y in zip(cs, ys):
        c.check(host(y))
    # in place, from a list
    ys = [c.dbase.clone() for c in cs]
    q().lora_add_batched([(c.table, None, y) for c, y in zip(cs, ys)], cs[0].dx, cs[0].dids, M, ws)
    for c, y in zip(cs, ys):
        c.check(host(y))


def test_workspace_is_not_written_past_its_size():
    for M, E in [(1, 1), (64, 3), (65, 2), (256, 300), (257, 300), (600, 2)]:
        c = Case("ws", M, 256, 64, 24, E, _ids("random", M, E))
        n = q().lora_ws(c.table, M)
        ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        c.check(c.run(ws=ws))
        assert (host(ws[n:]) == 0x5A).all()


@pytest.mark.parametrize("M", [1, 8, 300])
def test_captured_replayed_and_on_another_stream(M):
    c = Case("graph", M, 512, 128, 16, 4, _ids("random", M, 4))
    ws = torch.full((q().lora_ws(c.table, M),), 0xAB, dtype=torch.uint8, device="cuda")
    y = torch.empty((M, c.N), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q().lora_add(c.table, c.dx, c.dids, M, y, ws, base=c.dbase, stream=s)
    s.synchronize()
    eager = host(y)
    c.check(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q().lora_add(c.table, c.dx, c.dids, M, y, ws, base=c.dbase)
    for i in range(3):
        y.fill_(float("nan"))
        ws.fill_(i)
        graph.replay()
        np.testing.assert_array_equal(host(y).view(np.int32), eager.view(np.int32))
    # new ids in the same buffer reach the next replay
    c.ids = ((c.ids + 1) % 4).astype(np.int32)
    c.dids.copy_(dev_i32(c.ids))
    graph.replay()
    c.check(host(y))


def test_outputs_past_two_gigabytes():
    """Rows beyond the kernels' 31-bit offsets run as pieces of the call, one after the other."""
    M, K, N, R, E = 1100, 256, 1 << 19, 8, 2
    print(f"lora M={M} N={N}: y of {M * N * 4 / 2 ** 30:.1f} GiB", flush=True)
    g = synth.rng("gpu-lora", "large")
    A = synth.bf16_bits(g.standard_normal((E, R, K)) / np.sqrt(K))
    B = synth.bf16_bits(g.standard_normal((E, N, R)) / np.sqrt(R))
    x = synth.bf16_bits(g.standard_normal((M, K)))
    ids = _ids("random", M, E)
    ids[0], ids[M - 1] = 7, -1               # an id outside in the first piece only
    dx, dids, da, db = dev_bf16(x), dev_i32(ids), dev_bf16(A), dev_bf16(B)
    L = q().lora_table(E, R, N, K, da, db, dev_f32(np.ones(E)))
    ws = torch.empty(q().lora_ws(L, M), dtype=torch.uint8, device="cuda")
    y = torch.ones((M, N), device="cuda")
    q().lora_add(L, dx, dids, M, y, ws)
    assert int(host(ws[:4].view(torch.int32))[0]) == 1
    per = (1 << 31) // (4 * N)
    rows = [0, 1, per - 1, per, per + 1, M - 2, M - 1]
    cols = np.r_[0:64, N // 2:N // 2 + 64, N - 64:N]
    got = host(y[rows][:, torch.from_numpy(cols).cuda()])
    want, mag = oracle.lora_ref(synth.bf16_to_f32(x[rows]), synth.bf16_to_f32(A), synth.bf16_to_f32(B[:, cols]),
                                np.ones(E), ids[rows], np.ones((len(rows), len(cols))))
    assert (np.abs(got - want) <= 2.0 ** -23 * ((K + 3 * R + 80) * mag + 1 + np.abs(want))).all()
    dids.fill_(-1)
    q().lora_add(L, dx, dids, M, y, ws)
    assert int(host(ws[:4].view(torch.int32))[0]) == 0


@pytest.mark.parametrize("E,kind", [(1, "one"), (2, "each"), (3, "some"), (6, "random"), (15, "each"), (40, "each")])
@pytest.mark.parametrize("M", [16, 31, 32, 47, 64])
def test_tiles_of_few_and_of_many_adapters(M, E, kind):
    """Both ways in which a wave finds its tile, with tiles that fill up and that do not."""
    c = Case("tiles", M, 256, 64, 8, E, _ids(kind, M, E, seed=M))
    c.check(c.run())
    c.check(c.run(in_place=True))


@pytest.mark.parametrize("M", [1794, 1025])
def test_uneven_pieces_stay_inside_the_workspace_and_agree(M):
    """Calls cut at 2^31 bytes of y: nothing past the workspace is written, and a row has the same bits
    in whichever piece it lies."""
    K, N, R, E = 4096, 1 << 19, 64, 2
    print(f"lora M={M} N={N}: y of {M * N * 4 / 2 ** 30:.1f} GiB", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M)
    da = (torch.randn((E, R, K), device="cuda", generator=g) / 64).bfloat16()
    db = torch.randn((E, N, R), device="cuda", generator=g).bfloat16() / 8
    L = q().lora_table(E, R, N, K, da, db, dev_f32(np.ones(E)))
    dx = torch.randn((1, K), device="cuda", generator=g).bfloat16().repeat(M, 1)
    dids = dev_i32(np.arange(M) % E)
    size = q().lora_ws(L, M)
    ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    y = torch.zeros((M, N), device="cuda")
    q().lora_add(L, dx, dids, M, y, ws[:size])
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0x5A).all())
    assert float(y[0].abs().max()) > 0
    for m0 in range(0, M, 200):
        part = y[m0:m0 + 200].view(torch.int32)
        for m in range(part.shape[0]):
            assert torch.equal(part[m], y[(m0 + m) % E].view(torch.int32)), m0 + m


class Many(Case):
    """A case of many rows: the reference of a whole adapter's rows at once (the same sums as
    oracle.lora_ref, which forms them row by row)."""

    def ref(self):
        x = synth.bf16_to_f32(self.x).astype(np.float64)
        y, mag = self.base.astype(np.float64), np.zeros(self.base.shape)
        for e in np.unique(self.ids[(self.ids >= 0) & (self.ids < self.E)]):
            mine = self.ids == e
            r = self.R if self.ranks is None else min(max(int(self.ranks[e]), 0), self.R)
            a, b = self.A[e, :r].astype(np.float64), self.B[e, :, :r].astype(np.float64)
            s = float(self.scale[e])
            y[mine] += s * (x[mine] @ a.T @ b.T)
            mag[mine] = abs(s) * (np.abs(x[mine]) @ np.abs(a).T @ np.abs(b).T)
        return y, mag

    def tiles(self, ws):
        """(adapter, rows) of each tile that the last call made, from its workspace: the tiles follow the
        header and the places of the rows.  Records past the tiles keep the workspace's stale bytes."""
        groups = min(self.M, self.E + 1)
        at = (256 + 4 * (self.M + 64 * (groups + 7)) + 255) // 256 * 256
        rec = host(ws)[at:at + 8 * (self.M // 16 + groups + 7)].view(np.int32).reshape(-1, 2)
        rec = rec[(rec[:, 1] > 0) & (rec[:, 0] >= -1)]
        assert rec[:, 1].sum() == self.M
        want = np.where((self.ids >= 0) & (self.ids < self.E), self.ids, -1)
        for e in np.unique(want):
            assert rec[rec[:, 0] == e, 1].sum() == (want == e).sum()
        return rec

    def run_tiles(self, in_place=False):
        """run(), and the most rows of a tile; nothing past the workspace may change."""
        n = q().lora_ws(self.table, self.M)
        ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
        y = self.run(in_place, ws)
        assert (host(ws[n:]) == 0xAB).all()
        return y, int(self.tiles(ws)[:, 1].max())


def test_the_reference_of_many_rows():
    c = Many("many", 40, 256, 64, 16, 3, _ids("some", 40, 3), ranks=[16, 0, 5])
    for a, b in zip(c.ref(), Case.ref(c)):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("M,K,E,kind,R", [
    (2049, 256, 3, "random", 8), (2080, 256, 3, "random", 16), (3000, 256, 5, "some", 32), (4096, 256, 1, "one", 64),
    (4095, 256, 7, "runs", 128), (2100, 512, 4, "random", 200), (2500, 256, 6, "random", 256), (513, 9728, 2, "random", 64),
    (700, 9728, 3, "runs", 16), (1100, 9728, 4, "some", 72)])
def test_tiles_of_64_rows(M, K, E, kind, R):
    """Enough rows an adapter that tiles hold up to 64: every rank variant, pieces of 16 that are full, in
    part and not at all."""
    c = Many("tile64", M, K, 160, R, E, _ids(kind, M, E))
    y, rows = c.run_tiles()
    assert 48 < rows <= 64
    c.check(y)
    z, _ = c.run_tiles(in_place=True)
    np.testing.assert_array_equal(y.view(np.int32), z.view(np.int32))
    assert c.flag == 0


@pytest.mark.parametrize("R", [72, 256])
def test_tiles_of_64_rows_with_ranks_of_each_adapter(R):
    M, E = 2600, 12
    ranks = [0, 1, 7, 8, 9, 31, 33, 63, 64, 65, 71, R]
    c = Many("tile64 mixed", M, 256, 96, R, E, _ids("some", M, E), ranks, pad=24, garbage=True)
    y, rows = c.run_tiles()
    assert 48 < rows <= 64
    c.check(y)


def test_tiles_of_64_rows_ids_outside():
    M, E = 2200, 4
    ids = _ids("random", M, E)
    ids[[0, 3, 2199]] = [4, -2, -2 ** 31]
    ids[1000:1070] = 2 ** 31 - 1
    c = Many("tile64 outside", M, 256, 64, 8, E, ids)
    y, rows = c.run_tiles()
    assert rows == 64 and c.flag == 1
    c.check(y)


@pytest.mark.parametrize("M,R", [(2300, 32), (4096, 256)])
def test_tiles_of_64_rows_a_rows_bits_depend_on_its_own_inputs_only(M, R):
    c = Many("tile64 bits", M, 256, 96, R, 6, _ids("random", M, 6))
    y0, rows = c.run_tiles()
    assert 48 < rows <= 64
    c.check(y0)
    np.testing.assert_array_equal(c.run().view(np.int32), y0.view(np.int32))
    p = np.random.default_rng(3).permutation(M)
    c.dx, c.dids, c.dbase = dev_bf16(c.x[p]), dev_i32(c.ids[p]), dev_f32(c.base[p])
    np.testing.assert_array_equal(c.run().view(np.int32), y0[p].view(np.int32))
    ids = (c.ids + 1) % 6
    ids[7] = c.ids[7]
    c.dx, c.dids, c.dbase = dev_bf16(c.x), dev_i32(ids), dev_f32(c.base)
    np.testing.assert_array_equal(c.run()[7].view(np.int32), y0[7].view(np.int32))


@pytest.mark.parametrize("ranks", [(16, 40, 128), (8, 256, 64)])
def test_tiles_of_64_rows_batched(ranks):
    M = 2300
    ids = _ids("some", M, 5)
    cs = [Many(f"tile64 qkv{i}", M, 256, n, r, 5, ids) for i, (n, r) in enumerate(zip((256, 64, 96), ranks))]
    for c in cs[1:]:
        c.x, c.dx = cs[0].x, cs[0].dx
    ys = [torch.full((M, c.N), float("nan"), device="cuda") for c in cs]
    jobs = q().lora_jobs([(c.table, c.dbase, y) for c, y in zip(cs, ys)])
    n = q().lora_batched_ws(jobs, M)
    ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    print(f"lora batched M={M}", flush=True)
    q().lora_add_batched(jobs, cs[0].dx, cs[0].dids, M, ws)
    assert 48 < int(cs[0].tiles(ws)[:, 1].max()) <= 64 and (host(ws[n:]) == 0xAB).all()
    for c, y in zip(cs, ys):
        c.check(host(y))


def test_tiles_of_64_rows_captured_and_replayed():
    M = 2300
    c = Many("tile64 graph", M, 256, 128, 72, 4, _ids("random", M, 4))
    eager, rows = c.run_tiles()
    assert 48 < rows <= 64
    c.check(eager)
    ws = torch.full((q().lora_ws(c.table, M),), 0xAB, dtype=torch.uint8, device="cuda")
    y = torch.empty((M, c.N), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q().lora_add(c.table, c.dx, c.dids, M, y, ws, base=c.dbase)
    for i in range(3):
        y.fill_(float("nan"))
        ws.fill_(i)
        graph.replay()
        np.testing.assert_array_equal(host(y).view(np.int32), eager.view(np.int32))


@pytest.mark.parametrize("M,E,kind", [(4096, 1500, "random"), (4096, 4096, "each"), (4096, 4096, "random"), (4095, 1023, "some"),
                                      (4096, 1024, "each"), (1100, 4096, "random"), (65, 4096, "some"), (3000, 130, "runs")])
def test_route_of_many_adapters(M, E, kind):
    """The route at its most rows and adapters: every row in one tile of its adapter, once."""
    c = Many("route", M, 256, 32, 8, E, _ids(kind, M, E))
    y, _ = c.run_tiles()
    c.check(y)
    assert c.flag == 0


@pytest.mark.parametrize("M,K,N", [(1100, 256, 1 << 19), (1100, 1 << 20, 32)])
def test_the_border_of_pieces(M, K, N):
    """Calls cut at 2^31 bytes of y, and of x: the rows on both sides of every border."""
    R, E = 8, 2
    print(f"lora M={M} K={K} N={N}: x of {M * K / 2 ** 29:.1f} GiB, y of {M * N / 2 ** 28:.1f} GiB", flush=True)
    g = torch.Generator(device="cuda").manual_seed(K)
    dx = torch.randn((M, K), device="cuda", generator=g, dtype=torch.bfloat16)
    da = torch.randn((E, R, K), device="cuda", generator=g, dtype=torch.bfloat16) / K ** 0.5
    db = torch.randn((E, N, R), device="cuda", generator=g, dtype=torch.bfloat16)
    ids = _ids("random", M, E)
    ids[[0, M - 1]] = [7, -1]
    L = q().lora_table(E, R, N, K, da, db, dev_f32(np.array([1.0, 0.5])))
    ws = torch.empty(q().lora_ws(L, M), dtype=torch.uint8, device="cuda")
    y = torch.ones((M, N), device="cuda")
    q().lora_add(L, dx, dev_i32(ids), M, y, ws)
    assert int(host(ws[:4].view(torch.int32))[0]) == 1
    at_most = (1 << 31) // max(2 * K, 4 * N)
    pieces = -(-M // at_most)
    per = -(-M // pieces)
    assert pieces == 2
    rows = sorted({r for b in range(0, M + 1, per) for r in range(b - 2, b + 3) if 0 <= r < M} | {M - 2, M - 1})
    cols = np.arange(N) if N < 256 else np.r_[0:64, N // 2:N // 2 + 64, N - 64:N]
    tc = torch.from_numpy(cols).cuda()
    got = host(y[rows][:, tc])
    want, mag = oracle.lora_ref(host(dx[rows].float()), host(da.float()), host(db[:, tc].float()), np.array([1.0, 0.5]),
                                ids[rows], np.ones((len(rows), len(cols))))
    assert (np.abs(got - want) <= 2.0 ** -23 * ((K + 3 * R + 80) * mag + 1 + np.abs(want))).all()


@pytest.mark.parametrize("M,E,R", [(1, 1, 8), (7, 2, 16), (64, 3, 72), (100, 3, 40), (300, 2, 256), (2100, 3, 24), (2100, 3, 256)])
def test_infinite_weights(M, E, R):
    """Where a weight of B is infinite the output is what the formula gives: infinite of the product's sign,
    NaN where infinities of both signs or 0 and an infinity meet, or where B holds NaN; the other outputs
    keep their values.  At most ranks u is two activations' sum times a power of two, a few bits long, so
    that its lower parts are 0."""
    c = Many("inf weights", M, 256, 96, R, E, _ids("random", M, E))
    g = np.random.default_rng(R)
    short = g.random(R) < 0.7
    short[0] = True
    c.A[:, short] = 0.0
    c.A[:, short, 0] = 1.0
    c.A[:, :, 5] = 1.0
    c.scale = (2.0 ** (np.arange(E) % 3 - 1)).astype(np.float32)
    x = synth.bf16_to_f32(c.x)
    x[g.random(M) < 0.5] = 1.0
    if M > 3:
        x[1] = 0.0
        x[3, 5] = np.inf
    c.x = (x.view(np.uint32) >> 16).astype(np.uint16)     # bf16 values as they are
    b = c.B
    b[:, 0, 0], b[:, 1, 0] = np.inf, -np.inf
    b[:, 2, 0], b[:, 2, R - 1] = np.inf, -np.inf
    b[:, 3, R - 1] = np.nan
    b[0, 95, R // 2] = np.inf
    c.dx = dev_bf16(c.x)
    c.table = q().lora_table(E, R, 96, 256, dev_bf16(synth.bf16_bits(c.A)),
                             dev_bf16((b.view(np.uint32) >> 16).astype(np.uint16)), dev_f32(c.scale))
    want, mag = c.base.astype(np.float64), np.zeros(c.base.shape)
    with np.errstate(invalid="ignore"):
        for e in range(E):
            mine = c.ids == e
            a, s, v = c.A[e].astype(np.float64), float(c.scale[e]), x[mine].astype(np.float64)
            u, u_mag = (v[:, None] * a).sum(-1), (np.abs(v)[:, None] * np.abs(a)).sum(-1)
            for r in range(R):
                want[mine] += s * u[:, r, None] * b[e, :, r]
                mag[mine] += s * u_mag[:, r, None] * np.abs(b[e, :, r])
    y = c.run()
    np.testing.assert_array_equal(np.isnan(y), np.isnan(want))
    wild = np.isinf(want)
    assert wild.any()
    np.testing.assert_array_equal(y[wild], want[wild])
    fine = np.isfinite(want)
    with np.errstate(invalid="ignore"):
        tol = 2.0 ** -23 * ((c.K + 3 * c.R + 80) * mag + np.abs(c.base) + np.abs(want))
        assert (np.abs(y - want)[fine] <= tol[fine]).all()
