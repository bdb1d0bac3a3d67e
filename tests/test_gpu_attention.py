"""Attention over the paged cache (q4nx_attention) against float64, row by row.

With off = |scale| sum |q_i k_i| + |s| of the largest key, a score is off by at most (D + 8) 2^-24 off (D products,
exact in fp32, added in some order, and a few roundings), its exponential by as much, by 2^-22 of its own (the
instruction, the subtraction's rounding at scores near the maximum) and by 2^-22 for each 32 keys that may rescale it;
weights are rounded to bf16 (2^-8 with a half step) in the numerator, n of them are added in fp32, and the result is
rounded to bf16:
  |out - ref| <= sum p|v| (2 d + 2^-8 + (n + 64) 2^-24) + 2^-8 |ref| + 2^-133,
  d = 2 (D + 8) 2^-24 off + 2^-22 (4 + n / 32)      (numerator and denominator: 2 d)
  |lse - ref| <= d + (n + 64) 2^-24 + 2^-22 (1 + |ref|).
"""
import numpy as np
import pytest

import oracle
import synth

from _gpu import dev_bf16, dev_f32, dev_i32, have_gpu, host, q, torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


class Case:
    """A cache of random pages, sequences that lie anywhere in it, and their rows."""

    def __init__(self, tag, q_len, kv_len, prefix=0, H=8, KH=2, D=128, page=64, kind="bf16", extra_rows=0, sharp=2.0,
                 max_q=None, spare_cols=1, first_row=0):
        g = self.g = synth.rng("gpu-attention", tag, *q_len[:8], *kv_len[:8], prefix, H, KH, D, page, kind)
        self.n, self.H, self.KH, self.D, self.page, self.kind = len(q_len), H, KH, D, page, kind
        self.kv_len, self.prefix = list(kv_len), prefix
        self.q_start = first_row + np.concatenate([[0], np.cumsum(q_len)])
        self.M = int(self.q_start[-1]) + extra_rows
        self.max_q = max(1, max(q_len)) if max_q is None else max_q
        self.cols = max(1, -(-max(kv_len) // page)) + spare_cols
        shared = -(-prefix // page)
        pages = self.pages = self.n * self.cols + shared + 1
        order = g.permutation(pages)
        self.table, self.shared = order[: self.n * self.cols].reshape(self.n, self.cols), order[self.n * self.cols : -1]
        self.x = {}
        for name in "kv":
            if kind == "bf16":
                self.x[name] = synth.bf16_bits(g.standard_normal((pages, KH, page, D)))
            else:
                self.x[name] = np.clip(np.rint(40 * g.standard_normal((pages, KH, page, D))), -127, 127).astype(np.int8)
                self.x[name + "s"] = ((0.5 + g.random((pages, KH, page))) / 40).astype(np.float32)
        self.q = synth.bf16_bits(sharp * g.standard_normal((self.M, H, D)))
        self.scale = D ** -0.5

    def spoil(self, value=None):
        """What no row may see: tokens behind the lengths, spare pages and the last page, as NaN and infinities."""
        used = np.zeros((self.pages, self.page), bool)
        for s, L in enumerate(self.kv_len):
            for t in range(L):
                used[self.table[s, t // self.page], t % self.page] = True
        for t in range(self.prefix):
            used[self.shared[t // self.page], t % self.page] = True
        bad = ~used
        if self.kind == "bf16":
            marks = np.array([0x7FC0, 0x7F80, 0xFF80, 0xFFFF], np.uint16)
            for name in "kv":
                x = self.x[name].transpose(0, 2, 1, 3)
                x[bad] = marks[self.g.integers(0, 4, x[bad].shape)]
        else:
            for name in ("ks", "vs"):
                x = self.x[name].transpose(0, 2, 1)
                x[bad] = np.array([np.nan, np.inf, -np.inf], np.float32)[self.g.integers(0, 3, x[bad].shape)]

    def upload(self):
        self.dq = dev_bf16(self.q)
        if self.kind == "bf16":
            self.dk, self.dv, ks, vs = dev_bf16(oracle.pack_k(self.x["k"])), dev_bf16(oracle.pack_v(self.x["v"])), None, None
        else:
            self.dk, self.dv = (torch.from_numpy(p(self.x[n])).cuda() for p, n in ((oracle.pack_k, "k"), (oracle.pack_v, "v")))
            ks, vs = dev_f32(self.x["ks"]), dev_f32(self.x["vs"])
        self.cache = q().kv_cache(self.KH, self.D, self.page, self.pages, self.dk, self.dv, k_scale=ks, v_scale=vs)
        self.dstart, self.dlen, self.dtable = dev_i32(self.q_start), dev_i32(self.kv_len), dev_i32(self.table)
        self.batch = q().attn_batch(self.dstart, self.dlen, self.dtable, self.max_q, prefix_len=self.prefix,
                                    prefix_pages=dev_i32(self.shared) if self.prefix else None)
        self.ws = torch.full((q().attention_ws(self.cache, self.batch, self.H, self.M),), 0xFF, dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.M, self.H, self.D), 0x1234, dtype=torch.int16, device="cuda")
        self.lse = torch.full((self.M, self.H), -77.0, device="cuda")
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def run(self, stream=None):
        q().attention(self.cache, self.batch, self.dq, self.H, self.M, self.scale, self.out, self.ws, lse=self.lse,
                      flags=self.flags, stream=stream)
        return self

    def _tokens(self, name, pages, n, h):
        x = self.x[name][pages[: -(-n // self.page)], h].reshape(-1, self.D)[:n]
        if self.kind == "bf16":
            return synth.bf16_to_f32(x).astype(np.float64)
        return x.astype(np.float64) * self.x[name + "s"][pages[: -(-n // self.page)], h].reshape(-1)[:n, None].astype(np.float64)

    def reference(self):
        own = lambda s, h: tuple(self._tokens(n, self.table[s], self.kv_len[s], h) for n in "kv")  # noqa: E731
        pre = lambda h: tuple(self._tokens(n, self.shared, self.prefix, h) for n in "kv")  # noqa: E731
        with np.errstate(invalid="ignore", over="ignore"):
            return oracle.attention_batch_ref(synth.bf16_to_f32(self.q).astype(np.float64), self.q_start, self.kv_len, own, pre,
                                              self.scale, self.H // self.KH)

    def check(self, ref=None, flags=0):
        out, lse, mag, off = self.reference() if ref is None else ref
        raw, glse = host(self.out).view(np.uint16), host(self.lse)
        got = synth.bf16_to_f32(raw).astype(np.float64)
        rows = ~np.isnan(lse[:, 0])
        n = self.prefix + np.array(max(self.kv_len))
        d = 2 * (self.D + 8) * 2.0 ** -24 * off + 2.0 ** -22 * (4 + n / 32)
        tol = mag * (2 * d[..., None] + 2.0 ** -8 + (n + 64) * 2.0 ** -24) + 2.0 ** -8 * np.abs(out) + 2.0 ** -133
        bad = ~(np.abs(got - out) <= tol) & rows[:, None, None]
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], out[bad][:4])
        none = np.isneginf(lse)
        assert (glse[none & rows[:, None]] == -np.inf).all()
        fine = rows[:, None] & ~none
        ltol = d + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(lse))
        assert (np.abs(glse[fine] - lse[fine]) <= ltol[fine]).all()
        # rows of no sequence are left as they were
        inside = np.zeros(self.M, bool)
        inside[self.q_start[0] : self.q_start[-1]] = True
        assert (raw[~inside] == 0x1234).all() and (glse[~inside] == -77.0).all()
        assert host(self.flags)[0] == flags
        return self


DIMS = [(8, 2, 128), (3, 3, 64), (7, 1, 64), (10, 2, 128), (4, 1, 256), (16, 1, 128), (20, 1, 64), (6, 2, 256)]


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("H,KH,D", DIMS)
@pytest.mark.parametrize("prefix", [0, 77])
def test_decode(kind, H, KH, D, prefix):
    """One row a sequence, at lengths around the borders of pages and tiles."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 300, 641]
    print(f"decode {kind} {H}/{KH} x {D} prefix {prefix}", flush=True)
    c = Case("decode", [1] * len(lens), lens, prefix, H, KH, D, 64 if D > 64 else 16, kind)
    c.spoil()
    c.upload().run().check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_pages(page, kind):
    lens = [1, 100, 1025, 500, 31]
    for prefix in (0, 1, 513):
        c = Case("pages", [1, 2, 1, 3, 1], lens, prefix, 4, 2, 64, page, kind)
        c.spoil()
        c.upload().run().check()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("q_len", [(2, 2, 2), (4, 1, 3), (5, 0, 8), (16, 16, 1), (0, 0, 1)])
@pytest.mark.parametrize("H,KH,D", [(8, 2, 128), (7, 1, 64), (5, 5, 128), (4, 2, 256)])
def test_windows(kind, q_len, H, KH, D):
    """A few rows a sequence, also of sequences no longer than their window, and of none."""
    for prefix, lens in ((0, [n + e for n, e in zip(q_len, (0, 70, 300))]), (130, [n + e for n, e in zip(q_len, (33, 0, 7))])):
        c = Case("window", list(q_len), lens, prefix, H, KH, D, 16, kind, extra_rows=2)
        c.spoil()
        c.upload().run().check()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("H,KH,D,page", [(4, 2, 128, 64), (3, 1, 64, 16), (2, 2, 256, 32), (9, 1, 128, 128)])
@pytest.mark.parametrize("q_len,more,prefix", [((40,), 0, 0), ((129,), 71, 0), ((100, 1, 257), 0, 65), ((64, 64), 200, 0), ((300,), 500, 190)])
def test_prompts(kind, H, KH, D, page, q_len, more, prefix):
    c = Case("prompt", list(q_len), [n + more for n in q_len], prefix, H, KH, D, page, kind, extra_rows=3)
    c.spoil()
    c.upload().run().check()


def test_long_prompt_and_long_cache():
    Case("long", [700], [3000], 1100, 2, 1, 128, 64, "bf16").upload().run().check()
    Case("long", [1, 1], [40000, 9], 0, 4, 1, 64, 64, "int8").upload().run().check()
    Case("long", [1, 2, 1], [5, 9, 11], 20011, 4, 1, 128, 16, "bf16").upload().run().check()


def test_many_sequences():
    g = synth.rng("many-seq")
    for n in (257, 1024):
        q_len = g.integers(0, 3, n).tolist()
        c = Case("many", q_len, [a + int(b) for a, b in zip(q_len, g.integers(0, 60, n))], 40, 2, 1, 64, 16, "bf16", extra_rows=5)
        c.spoil()
        c.upload().run().check()


@pytest.mark.parametrize("n_heads", [(1, 1), (256, 1), (64, 64)])
def test_many_and_few_heads(n_heads):
    H, KH = n_heads
    c = Case("heads", [3, 1, 40], [50, 9, 77], 33, H, KH, 64, 16)
    c.spoil()
    c.upload().run().check()


def test_rows_that_see_nothing():
    """No tokens at all, and windows longer than the cached tokens: rows before the first token see nothing."""
    c = Case("nothing", [1, 3, 2, 40], [0, 1, 0, 5], 0, 4, 2, 128, 16)
    c.spoil()
    c.upload().run().check()
    lse = host(c.lse)
    assert np.isneginf(lse[0]).all() and np.isneginf(lse[1:3]).all() and np.isfinite(lse[3]).all()
    assert (host(c.out)[:3] == 0).all()
    c = Case("nothing", [1, 3, 2], [0, 1, 0], 3, 4, 2, 128, 16)       # and with a prefix they see that
    c.spoil()
    c.upload().run().check()
    assert np.isfinite(host(c.lse)).all()


def test_rows_before_the_first_sequence():
    c = Case("offset", [2, 1], [30, 40], 20, 4, 2, 64, 16, first_row=5, extra_rows=4)
    c.upload().run().check()


@pytest.mark.parametrize("q_len,kv_len,H,KH", [([4, 3], [40, 3], 4, 2), ([150], [400], 2, 1), ([33, 1], [70, 9], 8, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_values_that_only_later_rows_see(q_len, kv_len, H, KH, D):
    """An infinity or NaN in a value reaches the rows that see its token, and no other; in a key likewise."""
    for what in ("v", "k"):
        c = Case("later", q_len, kv_len, 0, H, KH, D, 16)
        s, back = 0, q_len[0] // 2                                  # the token of the sequence's middle row
        tok = kv_len[s] - 1 - back
        for h in range(KH):
            c.x[what][c.table[s, tok // 16], h, tok % 16, 5] = [0x7F80, 0x7FC0, 0xFF80][h % 3]
        c.upload().run()
        clean = Case("later", q_len, kv_len, 0, H, KH, D, 16)
        ref = clean.reference()
        first = q_len[0] - 1 - back                                 # the first row that sees it
        got, lse = synth.bf16_to_f32(host(c.out).view(np.uint16)), host(c.lse)
        for name, arr in (("out", got), ("lse", lse)):
            assert np.isfinite(arr[:first]).all() and np.isfinite(arr[q_len[0]:]).all(), name
        hit = np.arange(first, q_len[0])
        if what == "v":
            assert not np.isfinite(got[hit][:, :, 5]).any()
            assert np.isfinite(np.delete(got[hit], 5, axis=2)).all() and np.isfinite(lse).all()
            keep = np.ones_like(got, bool)
            keep[hit, :, 5] = False
        else:
            keep = np.ones_like(got, bool)
            keep[hit] = False
        out, _, mag, off = ref
        d = 2 * (D + 8) * 2.0 ** -24 * off + 2.0 ** -22 * (4 + max(kv_len) / 32)
        tol = mag * (2 * d[..., None] + 2.0 ** -8 + (max(kv_len) + 64) * 2.0 ** -24) + 2.0 ** -8 * np.abs(out) + 2.0 ** -133
        assert (np.abs(got - out)[keep] <= tol[keep]).all()


def test_scores_out_of_the_ordinary():
    """Scores far apart, one key above all, a scale of 0, a negative one."""
    c = Case("sharp", [1, 20], [500, 90], 70, 4, 2, 64, 16, sharp=60.0)
    c.upload().run().check()
    for scale in (0.0, -0.3):
        c = Case("scale", [1, 20], [500, 90], 70, 4, 2, 64, 16)
        c.scale = scale
        c.upload().run().check()


def test_pages_outside_the_cache():
    """A bad page is never followed: its tokens count as unseen, and the flag tells."""
    for kind in ("bf16", "int8"):
        for page in (16, 64):
            for q_len in ([1, 2], [70, 1]):
                c = Case("bad", q_len, [200, 90], 40, 4, 2, 64, page, kind)
                c.upload()
                table = c.table.copy()
                table[0, 1], table[1, 0] = c.pages, -1
                table[:, -1] = 1 << 30                              # a spare column: never looked at
                c.dtable.copy_(torch.from_numpy(table.astype(np.int32)))
                c.run()
                keep = {s: np.delete(np.arange(n), np.arange(b * page, min((b + 1) * page, n)))
                        for s, (n, b) in enumerate(((200, 1), (90, 0)))}
                # the reference sees the other tokens, each at its place
                out, lse, mag, off = (np.full(s, np.nan) for s in ((c.M, 4, 64), (c.M, 4), (c.M, 4, 64), (c.M, 4)))
                qv = synth.bf16_to_f32(c.q).astype(np.float64)
                for s in range(2):
                    for m in range(c.q_start[s], c.q_start[s + 1]):
                        see = c.kv_len[s] - q_len[s] + (m - c.q_start[s]) + 1
                        idx = keep[s][keep[s] < see]
                        for h in range(4):
                            k, v = (np.concatenate([c._tokens(n, c.shared, 40, h // 2), c._tokens(n, c.table[s], c.kv_len[s], h // 2)[idx]]) for n in "kv")
                            out[m, h], lse[m, h], mag[m, h], off[m, h] = oracle.attention_ref(qv[m, h], k, v, c.scale)
                c.check((out, lse, mag, off), flags=1)


def test_lengths_that_do_not_fit():
    """Too long a kv_len and falling starts are clamped, and the flag tells."""
    c = Case("clamp", [1, 2, 1], [40, 64, 20], 0, 4, 2, 64, 16, extra_rows=2, spare_cols=0)
    c.upload()
    c.dlen.copy_(torch.tensor([40, 9999, 20], dtype=torch.int32))   # four pages of 16 are 64 tokens
    c.run().check(flags=2)
    c.dlen.copy_(torch.tensor([-5, 64, 20], dtype=torch.int32))
    c.flags.zero_()
    c.kv_len[0] = 0
    c.run().check(flags=2)
    c = Case("clamp", [2, 0, 3], [40, 9, 64], 0, 4, 2, 64, 16, extra_rows=0)
    c.upload()
    c.dstart.copy_(torch.tensor([0, 2, 1, 99], dtype=torch.int32))  # falls, then passes the rows
    c.run().check(flags=2)


def test_captured_with_lengths_that_grow():
    """One graph over a growing cache, replayed between eager calls, each replay against the eager result."""
    c = Case("graph", [1, 1, 2], [300, 40, 90], 100, 8, 2, 128, 16)
    c.upload()
    eager = Case("graph", [1, 1, 2], [300, 40, 90], 100, 8, 2, 128, 16).upload()
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for lens in ([300, 40, 90], [299, 17, 2], [5, 31, 33], [300, 1, 64]):
        for x in (c, eager):
            x.dlen.copy_(torch.tensor(lens, dtype=torch.int32))
            x.kv_len = lens
            x.out.fill_(7)
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, eager.out) and torch.equal(c.lse, eager.lse)
    c.check()


def test_two_calls_on_two_streams_and_twice_the_same_bits():
    cs = [Case("stream", [1] * 9, [50 + 40 * i for i in range(9)], 300 + i, 8, 2, 64, 16).upload() for i in range(2)]
    for c in cs:
        c.run().check()
    first = [c.out.clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, want in zip(cs, first):
        assert torch.equal(c.out, want)


def test_offsets_past_two_and_four_billion_elements():
    """The last pages of a cache of 2^32 elements and more."""
    KH, D, page = 8, 128, 1024
    pages = (1 << 32) // (KH * D * page) + 2
    k, v = (torch.zeros(pages * KH * D * page, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages * KH * page,), 0.01, device="cuda") for _ in range(2))
    c = Case("far", [1, 2], [1500, 700], 0, 16, KH, D, page, "int8")
    for name, t, pack in (("k", k, oracle.pack_k), ("v", v, oracle.pack_v)):
        t.view(pages, -1)[-c.pages:] = torch.from_numpy(pack(c.x[name])).cuda().view(c.pages, -1)
    for name, t in (("ks", ks), ("vs", vs)):
        t.view(pages, -1)[-c.pages:] = dev_f32(c.x[name]).view(c.pages, -1)
    c.upload()
    c.cache = q().kv_cache(KH, D, page, pages, k, v, k_scale=ks, v_scale=vs)
    c.dtable += pages - c.pages
    c.run().check()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("max_q", [1, 5, 17, 40, 60000])
def test_max_q_is_a_hint(kind, max_q):
    """Whichever kernels max_q leads to, every row is computed."""
    for prefix in (0, 100):
        c = Case("hint", [1, 40, 3, 150], [90, 41, 200, 150], prefix, 4, 1, 64, 16, kind, max_q=max_q, extra_rows=2)
        c.spoil()
        c.upload().run().check()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("H,KH,D", [(8, 2, 128), (4, 4, 64), (6, 2, 256)])
@pytest.mark.parametrize("q_len", [(1,) * 40, (4,) * 9, (9,) * 9, (1, 12, 0, 7)])
def test_shared_prefix(kind, H, KH, D, q_len):
    """Enough rows together that the prefix's kernel has tiles of its own, of 16, 32 and 128 rows."""
    print(f"shared {kind} {H}/{KH} x {D}, rows {q_len}", flush=True)
    for prefix in (40, 700):
        c = Case("shared", list(q_len), [n + 13 * i % 90 for i, n in enumerate(q_len)], prefix, H, KH, D, 16, kind, extra_rows=1)
        c.spoil()
        c.upload().run().check()


def test_prefix_alone():
    """Sequences without tokens of their own, behind a prefix: their rows see it and nothing else."""
    c = Case("alone", [1, 2, 1], [0, 0, 0], 333, 4, 2, 64, 16)
    c.spoil()
    c.upload().run().check()


def test_values_that_only_later_rows_see_among_many_sequences():
    """The same behind a shared prefix, for windows and for prompts, and in the first and the last tokens."""
    for q_len, kv_len in (([4] * 6, [20] * 6), ([70, 90], [70, 300])):
        for back in (0, q_len[0] - 1):
            c, clean = (Case("later2", q_len, kv_len, 50, 4, 1, 64, 16) for _ in range(2))
            tok = kv_len[0] - 1 - back
            c.x["v"][c.table[0, tok // 16], 0, tok % 16, :9] = 0xFF80
            c.spoil()
            c.upload().run()
            first = q_len[0] - 1 - back
            got = synth.bf16_to_f32(host(c.out).view(np.uint16))
            assert not np.isfinite(got[first:q_len[0], :, :9]).any()
            out, _, mag, off = clean.reference()
            keep = np.ones_like(got, bool)
            keep[first:q_len[0], :, :9] = False
            d = 2 * (64 + 8) * 2.0 ** -24 * off + 2.0 ** -22 * (4 + (max(kv_len) + 50) / 32)
            tol = mag * (2 * d[..., None] + 2.0 ** -8 + (max(kv_len) + 114) * 2.0 ** -24) + 2.0 ** -8 * np.abs(out) + 2.0 ** -133
            assert (np.abs(got - out)[keep] <= tol[keep]).all()


def test_without_lse_and_flags():
    for q_len, kv_len in (([1, 1], [300, 9]), ([90], [500])):
        c = Case("bare", q_len, kv_len, 30, 4, 2, 64, 16).upload().run()
        want = c.out.clone()
        c.out.zero_()
        q().attention(c.cache, c.batch, c.dq, c.H, c.M, c.scale, c.out, c.ws)
        assert torch.equal(c.out, want)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("q_len", [(1, 1, 1), (20, 3, 70)])
def test_a_page_several_times(kind, q_len):
    """Pages that sequences share, one twice in a sequence, and one that is the prefix's too."""
    c = Case("shared-pages", q_len, [200, 170, 150], 40, 8, 2, 128, 32, kind)
    c.table[1, :3] = c.table[0, :3]
    c.table[2, 1] = c.table[2, 0]
    c.table[2, 2] = c.shared[0]
    c.upload().run().check()


@pytest.mark.parametrize("q_len", [(1, 1), (90, 30)])
def test_two_graphs_that_share_a_workspace(q_len):
    """Captured apart, replayed in turn with eager calls of another shape on the same workspace between them."""
    cs = [Case("one-workspace", q_len, L, pre, 8, 2, 128, 16).upload() for L, pre in (([700, 90], 0), ([300, 555], 130))]
    other = Case("one-workspace-eager", [3], [400], 0, 8, 2, 128, 16).upload()
    ws = torch.empty(max(c.ws.numel() for c in (*cs, other)), dtype=torch.uint8, device="cuda")
    for c in (*cs, other):
        c.ws = ws
    graphs = []
    for c in cs:
        c.run().check()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    want = [(c.out.clone(), c.lse.clone()) for c in cs]
    for i in (0, 1, 1, 0, 1, 0, 0):
        cs[i].out.fill_(7)
        cs[i].lse.fill_(7)
        graphs[i].replay()
        other.run()
        assert torch.equal(cs[i].out, want[i][0]) and torch.equal(cs[i].lse, want[i][1])
    other.check()


def _scores(c):
    """Of each row and head the scores that it sees, in float64, and their values (prefix first)."""
    qv = synth.bf16_to_f32(c.q).astype(np.float64)
    for s in range(c.n):
        for kh in range(c.KH):
            k, v = (np.concatenate([c._tokens(n, c.shared, c.prefix, kh), c._tokens(n, c.table[s], c.kv_len[s], kh)]) for n in "kv")
            for m in range(c.q_start[s], c.q_start[s + 1]):
                see = c.prefix + c.kv_len[s] - (c.q_start[s + 1] - m) + 1
                for h in range(kh * (c.H // c.KH), (kh + 1) * (c.H // c.KH)):
                    off = abs(c.scale) * (np.abs(k[:see]) @ np.abs(qv[m, h])).max()
                    yield m, h, c.scale * (k[:see] @ qv[m, h]), v[:see], off


def _far_scores(kind, scale, q_len, more, prefix, D):
    """Scores so large that one key has all the weight: its value comes out, whichever kernel the rows take.

    A score is off by at most (D + 8) 2^-24 sum |q_i k_i|; where the largest is further than twice that and 200 above
    the next, every other weight is below 2^-288 and 0 in fp32.  The value is then off by a bf16 weight's and the output's
    rounding, 2^-8 each; lse by its score's error and fp32's rounding."""
    c = Case("far-scores", list(q_len), [n + more for n in q_len], prefix, 4, 2, D, 16, kind)
    c.scale = scale
    c.upload().run()
    got, lse = synth.bf16_to_f32(host(c.out).view(np.uint16)).astype(np.float64), host(c.lse).astype(np.float64)
    assert np.isfinite(got).all() and np.isfinite(lse).all()
    alone = rows = 0
    for m, h, s, v, off in _scores(c):
        rows += 1
        err = (D + 8) * 2.0 ** -24 * off
        a, b = np.sort(s)[-1:-3:-1]
        assert abs(lse[m, h] - a) <= err + np.log(len(s)) + 2.0 ** -22 * abs(a)
        if a - b <= 2 * err + 200:
            continue
        alone += 1
        want = v[np.argmax(s)]
        assert (np.abs(got[m, h] - want) <= 2.1 * 2.0 ** -8 * np.abs(want)).all()
    assert alone > rows / 2


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("scale", [2.0 ** 18, 2.0 ** 31, -(2.0 ** 34), 1e36])
@pytest.mark.parametrize("q_len,prefix,D", [((1, 3), 0, 128), ((1, 3), 40, 64), ((4,), 0, 128)])
def test_scores_far_from_zero_of_few_rows(kind, scale, q_len, prefix, D):
    _far_scores(kind, scale, q_len, 500, prefix, D)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("scale", [2.0 ** 18, 2.0 ** 22, 2.0 ** 28, 2.0 ** 31, -(2.0 ** 34), 2.0 ** 80, 1e36])
@pytest.mark.parametrize("q_len,more,prefix,D", [((150,), 250, 0, 128), ((70, 40), 30, 90, 64), ((40,), 9, 0, 256),
                                                 ((1,) * 40, 20, 300, 128), ((4,) * 9, 50, 200, 64)])
def test_scores_far_from_zero_of_many_rows(kind, scale, q_len, more, prefix, D):
    _far_scores(kind, scale, q_len, more, prefix, D)


def _even_keys(kind):
    """Scores at which bf16 rounds the weight exp(s) up by most of half a step, and down: (up, down)."""
    if kind == "bf16":
        s = synth.bf16_to_f32(synth.bf16_bits(-np.arange(300, 700) / 1024.0)).astype(np.float64)
    else:
        s = -np.arange(300, 700) / 1024.0
    e = np.exp(s)
    r = synth.bf16_to_f32(synth.bf16_bits(e)).astype(np.float64) / e - 1
    return s[np.argmax(r)], s[np.argmin(r)]


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("q_len,own,prefix", [((1,), 4001, 0), ((1, 1, 1), 700, 0), ((4, 2), 999, 0), ((8,), 300, 2000), ((1,) * 40, 20, 3000),
                                              ((4,) * 9, 40, 2777), ((1,) * 5, 100, 1000)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_few_rows_keep_sixteen_bits_of_their_weights(kind, q_len, own, prefix, D):
    """Sequences of up to 32 rows of a key head, with and without a prefix, however many they are together.

    Half of the keys have a weight that bf16 rounds up, half one that it rounds down, and their values cancel: weights of
    8 bits would be off by about 2^-8 sum p|v|, far past what is allowed here, where the second part's half step is
    2^-8 of the first's, 2^-8 of the weight:  |out - ref| <= sum p|v| (2 d + 2^-16 + (n + 64) 2^-24) + 2^-8 |ref| + 2^-133
    (d: above; 8 bits: one more rounding, of the weight times the value's scale).  One key of 16 has the largest score
    and a value of 0, so that every part of a row counts from the same maximum."""
    H, KH = 8, 2
    up, down = _even_keys(kind)
    c = Case("even", list(q_len), [n + own for n in q_len], prefix, H, KH, D, 16, kind)
    c.scale = 1.0
    c.q[:] = 0
    c.q[..., 0] = 0x3F80
    tok = np.arange(16)
    first, odd = tok == 0, tok % 2 == 1
    ratio = 8 * np.exp(up) / (7 * np.exp(down))
    for name in "kv":
        c.x[name][:] = 0
    if kind == "bf16":
        c.x["k"][..., 0] = synth.bf16_bits(np.where(first, 0.0, np.where(odd, up, down)))
        c.x["v"][:] = synth.bf16_bits(np.where(first, 0.0, np.where(odd, 1.0, -ratio)))[:, None]
    else:
        c.x["k"][..., 0] = np.where(first, 0, -1)
        c.x["ks"][:] = np.where(odd, -up, -down).astype(np.float32)
        c.x["v"][:] = np.where(first, 0, np.where(odd, 80, -np.rint(80 * ratio))).astype(np.int8)[:, None]
        c.x["vs"][:] = 1 / 64
    c.upload().run()
    out, lse, mag, off = c.reference()
    got = synth.bf16_to_f32(host(c.out).view(np.uint16)).astype(np.float64)
    n = prefix + own + max(q_len)
    d = 2 * (D + 8) * 2.0 ** -24 * off + 2.0 ** -22 * (4 + n / 32)
    tol = mag * (2 * d[..., None] + 2.0 ** -16 + (n + 65) * 2.0 ** -24) + 2.0 ** -8 * np.abs(out) + 2.0 ** -133
    assert tol.max() < 2.0 ** -10 * mag.max()                   # what this is for: a fourth of one bf16 part's error
    bad = ~(np.abs(got - out) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], out[bad][:4], tol[bad][:4])
    ltol = d + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(lse))
    assert (np.abs(host(c.lse) - lse) <= ltol).all()


@pytest.mark.parametrize("q_len", [(1, 1, 1), (3, 2, 90)])
def test_a_table_within_a_wider_one(q_len):
    """The first columns of a table whose others are pages of the cache as well."""
    for prefix in (0, 100):
        c = Case("wide-table", q_len, [200, 170, 150], prefix, 8, 2, 128, 16)
        c.upload()
        wide = torch.randint(0, c.pages, (3, c.cols + 9), dtype=torch.int32, device="cuda")
        wide[:, : c.cols] = c.dtable
        c.batch = q().attn_batch(c.dstart, c.dlen, wide[:, : c.cols], c.max_q, prefix_len=prefix,
                                 prefix_pages=dev_i32(c.shared) if prefix else None)
        assert c.batch.pages_ld == c.cols + 9
        c.run().check()


@pytest.mark.parametrize("q_len", [(1,) * 9, (3, 70, 150)])
def test_two_streams_write_every_row_each_time(q_len):
    """Calls that run beside each other, each behind a fill of its outputs, leave the same bits every time."""
    cs = [Case("stream-fill", q_len, [n + 50 + 40 * i for i, n in enumerate(q_len)], 300 + j, 8, 2, 64, 16).upload() for j in range(2)]
    for c in cs:
        c.run().check()
    want = [(c.out.clone(), c.lse.clone()) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                c.out.fill_(0x1234)
                c.lse.fill_(-77)
                c.ws.fill_(0xFF)
                c.run()
        torch.cuda.synchronize()
        for c, (out, lse) in zip(cs, want):
            assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
