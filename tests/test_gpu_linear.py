"""Linear attention with decay (q4nx_linear_attn) against the recurrence in float64.

Every term of an output or state is a product of exact bf16 values, a decay and a scale, added in fp32.  A decay over T
rows is at most T exponentials (each off by 2^-22) or one exponential of a sum formed in fp64 (2^-22); operands of the
chunks' products keep 24 bits (three bf16 parts, 2^-23); the sums over dk lines, T rows and the parts add at most
dk + T + 64 roundings:  |x - x_ref| <= (5 T + dk + 96) 2^-24 sum |terms| + 2^-130.
"""
import numpy as np
import pytest

import oracle
import synth

from _gpu import dev_bf16, dev_f32, dev_i32, have_gpu, host, q, torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


class Case:
    def __init__(self, tag, lens, KH=2, H=4, dk=128, dv=128, by_token=True, extra_rows=0, first_row=0, pad=0, speed=0.05,
                 max_q=None, fresh=None, slots=None):
        g = self.g = synth.rng("gpu-linear", tag, *lens[:8], KH, H, dk, dv, by_token)
        self.n, self.KH, self.H, self.dk, self.dv, self.lens = len(lens), KH, H, dk, dv, list(lens)
        self.q_start = first_row + np.concatenate([[0], np.cumsum(lens)])
        self.M = max(1, int(self.q_start[-1]) + extra_rows)
        self.max_q = max(1, max(lens)) if max_q is None else max_q
        M = self.M
        self.q, self.k, self.v = (synth.bf16_bits(s * g.standard_normal((M, n, d)))
                                  for n, d, s in ((KH, dk, 1), (KH, dk, dk ** -0.5), (H, dv, 1)))
        self.decay = (-speed * np.exp(g.standard_normal((M, H)) * 1.5)).astype(np.float32)
        self.by_token = by_token
        if not by_token:
            self.decay[:] = self.decay[0]
        self.n_slots = self.n + 3
        self.slots = g.permutation(self.n_slots)[: self.n] if slots is None else np.array(slots)
        self.fresh = fresh
        self.state = g.standard_normal((self.n_slots, H, dk, dv)).astype(np.float32)
        self.pad, self.scale = pad, dk ** -0.5

    def upload(self, in_place=False):
        def rows(x):
            flat = x.reshape(self.M, -1)
            t = dev_bf16(np.concatenate([flat, np.full((self.M, self.pad), 0x7FC0, np.uint16)], 1)) if self.pad else dev_bf16(flat)
            return t[:, : flat.shape[1]]
        self.dq, self.dk_, self.dv_ = rows(self.q), rows(self.k), rows(self.v)
        self.ddecay = dev_f32(self.decay if self.by_token else self.decay[0])
        self.dstart, self.dslots = dev_i32(self.q_start), dev_i32(self.slots)
        self.seqs = q().linear_attn_seqs(self.dstart, self.dslots, self.max_q, fresh=None if self.fresh is None else dev_i32(self.fresh))
        self.dstate = dev_f32(self.state)
        self.dstate_out = self.dstate if in_place else torch.full_like(self.dstate, -5.0)
        self.out = torch.full((self.M, self.H, self.dv), -9.0, device="cuda")
        self.ws = torch.full((q().linear_attn_ws(self.seqs, self.KH, self.H, self.dk, self.dv, self.M),), 0xFF, dtype=torch.uint8, device="cuda")
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def run(self, stream=None):
        q().linear_attn(self.seqs, self.dq, self.dk_, self.dv_, self.ddecay, self.KH, self.H, self.dk, self.dv, self.M, self.scale,
                        self.dstate, self.out, self.ws, state_out=self.dstate_out, flags=self.flags, stream=stream)
        return self

    def reference(self):
        out, mag = np.full((self.M, self.H, self.dv), np.nan), np.full((self.M, self.H, self.dv), np.nan)
        states = {}
        f = lambda x: synth.bf16_to_f32(x).astype(np.float64)  # noqa: E731
        taken = set()
        for s, n in enumerate(self.lens):
            slot = int(self.slots[s])
            if not 0 <= slot < self.n_slots or slot in taken:
                slot = -1
            if n and slot >= 0:
                taken.add(slot)
            r = slice(self.q_start[s], self.q_start[s + 1])
            begin = slot < 0 or (self.fresh is not None and self.fresh[s])
            new, amag = np.zeros((2, self.H, self.dk, self.dv))
            for h in range(self.H):
                kh = h // (self.H // self.KH)
                S = np.zeros((self.dk, self.dv)) if begin else self.state[slot, h]
                out[r, h], new[h], mag[r, h], amag[h] = oracle.linear_attn_ref(
                    f(self.q[r, kh]), f(self.k[r, kh]), f(self.v[r, h]), np.minimum(self.decay[r, h], 0), self.scale, S)
            if n and slot >= 0:
                states[slot] = (new, amag)
        return out, mag, states

    def check(self, flags=0, ref=None):
        out, mag, states = self.reference() if ref is None else ref
        c = (5 * max(self.lens) + self.dk + 96) * 2.0 ** -24
        got, state = host(self.out).astype(np.float64), host(self.dstate_out).astype(np.float64)
        rows = ~np.isnan(mag[:, 0, 0])
        bad = ~(np.abs(got - out) <= c * mag + 2.0 ** -130) & rows[:, None, None]
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], out[bad][:4], (c * mag)[bad][:4])
        inside = np.zeros(self.M, bool)
        inside[self.q_start[0] : self.q_start[-1]] = True
        assert (got[~inside] == -9.0).all()
        before = self.state if self.dstate_out is self.dstate else np.full_like(self.state, -5.0)
        for slot in range(self.n_slots):
            if slot not in states:
                np.testing.assert_array_equal(state[slot], before[slot].astype(np.float64))
                continue
            new, amag = states[slot]
            bad = ~(np.abs(state[slot] - new) <= c * amag + 2.0 ** -130)
            assert not bad.any(), (slot, bad.sum(), np.argwhere(bad)[:4], state[slot][bad][:4], new[bad][:4])
        assert host(self.flags)[0] == flags
        return self


SHAPES = [(1, 1, 64, 64), (2, 4, 128, 128), (3, 3, 64, 128), (2, 6, 128, 64)]


@pytest.mark.parametrize("KH,H,dk,dv", SHAPES)
@pytest.mark.parametrize("n", [1, 5, 130])
def test_one_token(KH, H, dk, dv, n):
    print(f"linear, {n} tokens, {KH}/{H} x {dk} x {dv}", flush=True)
    for in_place in (False, True):
        Case("one", [1] * n, KH, H, dk, dv, extra_rows=2).upload(in_place).run().check()


@pytest.mark.parametrize("KH,H,dk,dv", SHAPES)
@pytest.mark.parametrize("lens", [(2,), (63,), (64,), (65,), (3, 0, 17), (128, 1, 129), (200,), (0, 5)])
@pytest.mark.parametrize("by_token", [True, False])
def test_lengths(KH, H, dk, dv, lens, by_token):
    print(f"linear, rows {lens}, {KH}/{H} x {dk} x {dv}", flush=True)
    Case("lens", list(lens), KH, H, dk, dv, by_token, extra_rows=1).upload().run().check()


@pytest.mark.parametrize("T", [777, 1500])
def test_long(T):
    for speed in (0.001, 0.3):
        Case("long", [T, 31], 1, 2, 128, 128, speed=speed).upload(True).run().check()


def test_many_sequences():
    g = synth.rng("linear-many")
    Case("many", g.integers(0, 9, 300).tolist(), 1, 2, 64, 64, extra_rows=3).upload().run().check()
    Case("many", [1] * 1024, 1, 1, 64, 64).upload(True).run().check()
    Case("many", [90] * 70, 1, 1, 64, 64).upload(True).run().check()


def test_strides_and_offsets():
    Case("pad", [1, 70, 3], 2, 4, 64, 128, pad=8, first_row=3, extra_rows=2).upload().run().check()
    Case("pad", [1, 1], 2, 4, 64, 128, pad=24, first_row=1).upload(True).run().check()


@pytest.mark.parametrize("lens", [[1, 1, 1, 1], [1, 70, 130, 2], [65, 64, 3, 300]])
def test_fresh_and_no_slot(lens):
    """Sequences that begin with zeros though their slot holds NaN, and ones whose state is neither read nor kept."""
    c = Case("fresh", lens, 1, 2, 64, 64, fresh=[1, 0, 0, 1], slots=[2, -1, 0, 5])
    c.state[[2, 5]] = np.nan
    c.upload(True).run()
    c.state[[2, 5]] = 0.0
    ref = c.reference()
    got = host(c.dstate)
    c.state = np.where(np.isnan(got), got, c.state)
    c.check(ref=ref)


@pytest.mark.parametrize("lens", [[1, 1, 1], [80, 0, 3], [130, 66, 70]])
def test_bad_and_repeated_slots(lens):
    """A slot outside the states, and one that an earlier sequence with rows has, count as none."""
    c = Case("slots", lens, 1, 2, 64, 64, slots=[4, 4, 4])
    c.upload(True).run().check(flags=1)
    for bad in (6, -2, 2 ** 31 - 1, -2 ** 31):
        Case("slots", lens, 1, 2, 64, 64, slots=[bad, 1, 0]).upload(True).run().check(flags=1)
    Case("slots", [0, 1, 70], 1, 2, 64, 64, slots=[3, 3, 0]).upload(True).run().check()    # the first has no rows


@pytest.mark.parametrize("lens", [[1, 1], [100, 7], [200, 65]])
def test_decays_out_of_the_ordinary(lens):
    """0 keeps all, -inf and the type's lowest value forget all (an infinite state too), tiny ones count."""
    c = Case("decay", lens, 1, 2, 64, 64)
    low = np.finfo(np.float32).min
    c.decay[:] = np.resize(np.array([0.0, -1e-6, -np.inf, -1.0, 0.0, low, -30.0, -1e-4, -0.0, -90.0], np.float32), c.decay.shape)
    c.upload().run().check()
    c = Case("decay", lens, 1, 2, 64, 64)
    c.decay[:] = 0
    c.upload().run().check()
    c = Case("decay", lens, 1, 2, 64, 64)
    c.decay[:] = -np.inf
    c.state[:] = np.inf
    c.state[0] = np.nan
    c.upload().run().check()
    # what is no decay counts as 0, and the flag tells
    c = Case("decay", lens, 1, 2, 64, 64)
    c.decay[c.q_start[1] - 1, 1] = 0.5
    c.upload().run().check(flags=2)
    c = Case("decay", lens, 1, 2, 64, 64)
    c.decay[0, 0] = np.nan
    c.upload()
    c.decay[0, 0] = 0
    c.run().check(flags=2)


@pytest.mark.parametrize("n", [70, 200])
def test_values_that_only_later_rows_see(n):
    """An infinity or NaN of a later row's v, k or q reaches no row before it, nor another sequence."""
    for name in "qkv":
        c = Case("later", [n, 20], 1, 1, 64, 64)
        at = n - 9
        getattr(c, name)[at, 0, 3] = 0x7F80
        getattr(c, name)[at + 2, 0, 3] = 0x7FC0
        c.upload().run()
        got = host(c.out)
        clean = Case("later", [n, 20], 1, 1, 64, 64)
        out, mag, _ = clean.reference()
        for rows in (slice(0, at), slice(n, n + 20)):
            assert (np.abs(got[rows] - out[rows]) <= (5 * n + 64 + 96) * 2.0 ** -24 * mag[rows]).all(), name
        assert not np.isfinite(got[at]).all()


def test_rows_that_do_not_fit():
    c = Case("clamp", [3, 0, 4], 1, 2, 64, 64)
    c.upload()
    c.dstart.copy_(torch.tensor([0, 3, 1, 99], dtype=torch.int32))
    c.run().check(flags=4)


@pytest.mark.parametrize("lens", [[1] * 20, [100, 3, 66]])
def test_captured(lens):
    c, eager = (Case("graph", lens, 2, 4, 64, 128).upload(True) for _ in range(2))
    c.run()
    eager.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.dstate.copy_(eager.dstate)
    for _ in range(4):
        graph.replay()
        eager.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, eager.out) and torch.equal(c.dstate, eager.dstate)
        c.dq.neg_()
        eager.dq.neg_()


def test_two_streams():
    cs = [Case("stream", [70 + i, 200], 1, 2, 64, 64).upload() for i in range(2)]
    for c in cs:
        c.run().check()
    want = [(c.out.clone(), c.dstate_out.clone()) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, (o, st) in zip(cs, want):
        assert torch.equal(c.out, o) and torch.equal(c.dstate_out, st)


def test_a_prompt_in_pieces():
    """The same rows in one call, in two, and token by token end with the same state, within the bound."""
    whole = Case("pieces", [150], 1, 2, 64, 128, slots=[0]).upload(True).run().check()
    ref = whole.reference()
    for cuts in ([0, 70, 150], [0, 64, 65, 66, 150], list(range(0, 151, 15))):
        c = Case("pieces", [150], 1, 2, 64, 128, slots=[0]).upload(True)
        for a, b in zip(cuts, cuts[1:]):
            c.dstart.copy_(torch.tensor([a, b], dtype=torch.int32))
            c.run()
        c.check(ref=ref)


@pytest.mark.parametrize("lens,H", [([5000], 32), ([2600, 40, 1100], 8), ([700], 2)])
def test_in_place_and_apart_end_alike(lens, H):
    """The last segment's end goes where the first one's state is read from: same bits as with a state of its own."""
    a = Case("place", lens, H // 2, H, 64, 64, speed=0.002).upload(False).run()
    b = Case("place", lens, H // 2, H, 64, 64, speed=0.002).upload(True)
    for _ in range(3):
        b.dstate.copy_(a.dstate)
        b.run()
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out)
        for s in range(len(lens)):
            assert torch.equal(a.dstate_out[a.slots[s]], b.dstate[a.slots[s]])


@pytest.mark.parametrize("max_q", [1, 5, 13, 100, 300, 60000])
def test_max_q_is_a_hint(max_q):
    """Rows past max_q are computed all the same."""
    Case("hint", [1, 70, 9, 330], 1, 2, 64, 64, max_q=max_q).upload(True).run().check()


def test_all_rows_in_one_long_sequence_of_many():
    """One sequence has all the rows of a call that other shapes would share."""
    for lens in ([0] * 20 + [900] + [0] * 11, [1] * 40 + [500]):
        Case("uneven", lens, 1, 1, 64, 64).upload(True).run().check()


def test_scales():
    for scale in (0.0, -1.5, 1e-30):
        for n in (1, 100):
            c = Case("scale", [n], 1, 1, 64, 64)
            c.scale = scale
            c.upload().run().check()


@pytest.mark.parametrize("lens,H", [([700], 2), ([260, 5, 400], 4), ([3000], 32)])
@pytest.mark.parametrize("rate", [-0.01, -2.0, -100.0])
@pytest.mark.parametrize("what", ["state", "k", "v"])
def test_infinities_and_nans_that_no_decay_cuts_off(lens, H, rate, what):
    """They stay in the state however far it has decayed, as no single decay's exp is 0, over any number of segments;
    one of -Inf cuts them off."""
    f = lambda x: synth.bf16_to_f32(x).astype(np.float64)  # noqa: E731
    for mark, cut in ((0x7FC0, False), (0x7F80, False), (0xFF80, False), (0x7FC0, True), (0xFF80, True)):
        c = Case("kept", lens, H, H, 64, 64)
        c.decay[:] = rate
        slot, begin, end = c.slots[-1], c.q_start[-2], c.q_start[-1]
        if what == "state":
            c.state[slot, 1, 3, 5] = f(np.array([mark], np.uint16))[0]
        else:
            getattr(c, what)[begin + 9, 1, 3] = mark
        if cut:
            c.decay[begin + 150, 1] = -np.inf
        c.upload().run()
        r = slice(begin, end)
        with np.errstate(invalid="ignore"):
            out, S, _, _ = oracle.linear_attn_ref(f(c.q[r, 1]), f(c.k[r, 1]), f(c.v[r, 1]), c.decay[r, 1], c.scale, c.state[slot, 1])
        assert np.isfinite(out[-1]).all() == cut and not np.isfinite(out[9]).all()
        got, state = host(c.out), host(c.dstate_out)
        np.testing.assert_array_equal(np.isfinite(got[r, 1]), np.isfinite(out))
        np.testing.assert_array_equal(np.isfinite(state[slot, 1]), np.isfinite(S))
        np.testing.assert_array_equal(np.isnan(state[slot, 1]), np.isnan(S))
        got[r, 1] = state[slot, 1] = 0
        assert np.isfinite(got).all() and np.isfinite(state).all()
        assert host(c.flags)[0] == 0


@pytest.mark.parametrize("max_q", [4, 100, 300])
@pytest.mark.parametrize("start,clamped", [([0, 100, 50], [0, 100, 100]), ([0, 100, 107], [0, 100, 100]), ([-5, 0, 100], [0, 0, 100]),
                                           ([10, 5], [10, 10]), ([0, 3, 1, 99], [0, 3, 3, 99]), ([0, 40, -1, -1, 60], [0, 40, 40, 40, 60]),
                                           ([0] * 70 + [100, 99], [0] * 70 + [100, 100])])
def test_row_starts_that_do_not_fit_are_told(max_q, start, clamped):
    """Falling starts and such as leave the rows, of sequences without rows too, whichever kernels run."""
    lens = np.diff(clamped).tolist()
    c = Case("told", lens, 1, 2, 64, 64, max_q=max_q, first_row=clamped[0], extra_rows=100 - clamped[-1])
    c.upload().run().check()
    c.upload()
    c.dstart.copy_(torch.tensor(start, dtype=torch.int32))
    c.run().check(flags=4)


@pytest.mark.parametrize("KH,H", [(1, 2), (16, 32)])
def test_a_workspace_for_many_rows_holds_fewer(KH, H):
    """One workspace, sized for the largest batch, for shorter ones whose segments are cut otherwise."""
    seqs = Case("one-ws", [4096], KH, H, 64, 64).upload().seqs
    ws = torch.empty(q().linear_attn_ws(seqs, KH, H, 64, 64, 4096), dtype=torch.uint8, device="cuda")
    for lens in ([768], [769], [300], [1500, 41], [5]):
        c = Case("one-ws", lens, KH, H, 64, 64, max_q=4096).upload()
        assert len(lens) > 1 or c.ws.numel() <= ws.numel()
        guard = torch.full((ws.numel() + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        c.ws = guard[: ws.numel()] if len(lens) == 1 else c.ws
        c.run().check()
        assert (host(guard[ws.numel():]) == 0xFF).all()


@pytest.mark.parametrize("lens", [(1,) * 9, (70, 200), (700, 3)])
def test_two_streams_write_every_row_each_time(lens):
    """Calls that run beside each other, each behind a fill of its outputs, leave the same bits every time."""
    cs = [Case("stream-fill", [n + i for n in lens], 1, 2, 64, 64).upload() for i in range(2)]
    for c in cs:
        c.run().check()
    want = [(c.out.clone(), c.dstate_out.clone()) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                c.out.fill_(-9.0)
                c.dstate_out.fill_(-5.0)
                c.ws.fill_(0xFF)
                c.run()
        torch.cuda.synchronize()
        for c, (out, state) in zip(cs, want):
            assert torch.equal(c.out, out) and torch.equal(c.dstate_out, state)
