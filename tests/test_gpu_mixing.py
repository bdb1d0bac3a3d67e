"""The token mixing of a layer as it runs: q|k|v from one projection, the heads' norms, rotation and append, attention
behind a shared prefix, the output projection; and the same with linear attention and its states.

Each stage is checked against the float64 reference of its own inputs, which are the device's outputs of the stage
before; a decode step is captured in a graph and replayed between eager work, and steps run on two streams.
"""
import numpy as np
import pytest

import oracle
import synth

from _gpu import dev_bf16, dev_f32, dev_i32, dev_u8, have_gpu, host, q, torch, weight

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

E, H, KH, D, PAGE = 512, 8, 2, 64, 16
EPS, P = 1e-6, 45


def _gemm(w, x, y, M, ws):
    if M <= q().GEMV_MAX_M:
        q().gemv(w, x, y, M)
    else:
        for m in range(0, M, q().GEMM_MAX_M):
            q().gemm_block(w, x[m:], y[m:], min(q().GEMM_MAX_M, M - m), ws)


class Layer:
    """Three sequences behind a prefix of P tokens, with room for a prompt and some steps."""

    def __init__(self, kind, tag="layer"):
        g = self.g = synth.rng("gpu-mixing", tag, kind)
        rows = (H + 2 * KH) * D
        self.kind, self.rows = kind, rows
        self.wqkv = weight(dev_u8(synth.gen_q4_1(g, rows, E, zero="normal")), rows, E, "q4_1")
        self.o_chunks = synth.gen_q4_1(g, E, H * D, zero="normal")
        self.wo = weight(dev_u8(self.o_chunks), E, H * D, "q4_1")
        self.nq, self.nk = (dev_bf16(synth.bf16_bits(1 + 0.2 * g.standard_normal(D))) for _ in range(2))
        pages = self.pages = 40
        dt = torch.int16 if kind == "bf16" else torch.int8
        self.k, self.v = (torch.full((pages * KH * PAGE * D,), 0x7F, dtype=dt, device="cuda") for _ in range(2))
        ks, vs = (torch.full((pages * KH * PAGE,), float("nan"), device="cuda") for _ in range(2)) if kind == "int8" else (None, None)
        self.ks, self.vs = ks, vs
        self.cache = q().kv_cache(KH, D, PAGE, pages, self.k, self.v, k_scale=ks, v_scale=vs)
        order = g.permutation(pages)
        self.shared, self.table = order[:3], order[3:33].reshape(3, 10)
        self.freq = dev_f32(1e4 ** (-np.arange(D // 2) / (D // 2)))
        self.len = np.zeros(3, int)
        self.ws = torch.zeros(max(256, q().gemm_block_ws(self.wqkv), q().gemm_block_ws(self.wo)), dtype=torch.uint8, device="cuda")

    def buffers(self, M, max_q):
        f = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
        b = dict(qkv=f(M, self.rows), qh=torch.zeros((M, H * D), dtype=torch.int16, device="cuda"),
                 kh=torch.zeros((M, KH * D), dtype=torch.int16, device="cuda"), raw=f(M, (H + KH) * D), qr=torch.zeros((M, H, D), dtype=torch.int16, device="cuda"),
                 out=torch.zeros((M, H, D), dtype=torch.int16, device="cuda"), y=f(M, E), x=torch.zeros((M, E), dtype=torch.int16, device="cuda"),
                 pos=torch.zeros(M, dtype=torch.int32, device="cuda"), slots=torch.zeros(M, dtype=torch.int32, device="cuda"),
                 start=torch.zeros(4, dtype=torch.int32, device="cuda"), lens=torch.zeros(3, dtype=torch.int32, device="cuda"), M=M)
        b["batch"] = q().attn_batch(b["start"], b["lens"], dev_i32(self.table), max_q, prefix_len=P, prefix_pages=dev_i32(self.shared))
        b["rope"] = q().rope(self.freq, b["pos"], D)
        b["aws"] = torch.empty(q().attention_ws(self.cache, b["batch"], H, M), dtype=torch.uint8, device="cuda")
        return b

    def fill(self, b, q_len):
        """Positions, slots and lengths of each sequence's next q_len[s] tokens; rows behind them are padding."""
        pos, slots = [], []
        for s, n in enumerate(q_len):
            at = self.len[s] + np.arange(n)
            pos += list(P + at)
            slots += [self.table[s, t // PAGE] * PAGE + t % PAGE for t in at]
            self.len[s] += n
        pad = b["M"] - len(pos)
        b["pos"].copy_(torch.tensor(pos + [0] * pad, dtype=torch.int32))
        b["slots"].copy_(torch.tensor(slots + [-1] * pad, dtype=torch.int32))
        b["start"].copy_(torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32))
        b["lens"].copy_(torch.tensor(self.len, dtype=torch.int32))
        b["x"].copy_(dev_bf16(synth.gen_x(self.g, b["M"], E)).view(b["M"], E))

    def mix(self, b):
        """q|k|v, norms, append; without attention where there are no sequences (the prefix)."""
        M = b["M"]
        _gemm(self.wqkv, b["x"], b["qkv"], M, self.ws)
        b["raw"].copy_(b["qkv"][:, : (H + KH) * D])                         # heads of q and k, each a row of the norm
        heads = b["raw"].view(M, H + KH, D)
        q().add_rmsnorm(heads[:, :H].contiguous(), self.nq, M * H, D, EPS, b["qh"])
        q().add_rmsnorm(heads[:, H:].contiguous(), self.nk, M * KH, D, EPS, b["kh"])
        q().kv_append(self.cache, b["kh"], b["qkv"][:, (H + KH) * D:], b["slots"], M, rope=b["rope"], q=b["qh"], q_heads=H, q_out=b["qr"])

    def step(self, b):
        self.mix(b)
        q().attention(self.cache, b["batch"], b["qr"], H, b["M"], D ** -0.5, b["out"], b["aws"])
        _gemm(self.wo, b["out"], b["y"], b["M"], self.ws)

    def prefix(self):
        b = self.buffers(P, 1)
        b["pos"].copy_(torch.arange(P, dtype=torch.int32))
        b["slots"].copy_(torch.tensor([self.shared[t // PAGE] * PAGE + t % PAGE for t in range(P)], dtype=torch.int32))
        b["x"].copy_(dev_bf16(synth.gen_x(self.g, P, E)).view(P, E))
        self.mix(b)
        self.check_append(b, P)

    def cached(self, slots):
        """(k, v) of the slots as floats."""
        out = []
        for raw, scale, unpack, shape in ((self.k, self.ks, oracle.unpack_k, (self.pages, KH, PAGE // 16, D // 8, 16, 8)),
                                          (self.v, self.vs, oracle.unpack_v, (self.pages, KH, PAGE // 8, D, 8))):
            x = host(raw)
            x = synth.bf16_to_f32(x.view(np.uint16)).astype(np.float64) if self.kind == "bf16" else x.astype(np.float64)
            x = unpack(x.reshape(shape)).transpose(0, 2, 1, 3).reshape(-1, KH, D)[slots]
            if scale is not None:
                x = x * host(scale).reshape(self.pages, KH, PAGE).transpose(0, 2, 1).reshape(-1, KH)[slots][..., None].astype(np.float64)
            out.append(x)
        return out

    def check_append(self, b, n):
        """The first n rows: what was stored is what the stage before gave, turned."""
        pos, slots = host(b["pos"])[:n], host(b["slots"])[:n]
        kh = synth.bf16_to_f32(host(b["kh"]).view(np.uint16)).reshape(-1, KH, D)[:n]
        qh = synth.bf16_to_f32(host(b["qh"]).view(np.uint16)).reshape(-1, H, D)[:n]
        v = host(b["qkv"])[:n, (H + KH) * D:].reshape(n, KH, D)
        f = host(self.freq)
        (wk, mk), (wq, mq) = (oracle.rope_ref(x, pos, f, D, False) for x in (kh, qh))
        gk, gv = self.cached(slots)
        gq = synth.bf16_to_f32(host(b["qr"]).view(np.uint16))[:n]
        near = lambda got, want, mag: np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 5 * 2.0 ** -24 * mag + 2.0 ** -134  # noqa: E731
        assert near(gq, wq, mq).all()
        if self.kind == "bf16":
            assert near(gk, wk, mk).all() and near(gv, v, np.abs(v)).all()
        else:   # half a step of the scale, and the scale's rounding
            for got, want in ((gk, wk), (gv, v.astype(np.float64))):
                assert (np.abs(got - want) <= (0.5 + 1e-4) * np.abs(want).max(-1, keepdims=True) / 127).all()

    def check_attention(self, b, q_len):
        qr = synth.bf16_to_f32(host(b["qr"]).view(np.uint16)).astype(np.float64)
        own = [self.cached([self.table[s, t // PAGE] * PAGE + t % PAGE for t in range(self.len[s])]) for s in range(3)]
        pre = self.cached([self.shared[t // PAGE] * PAGE + t % PAGE for t in range(P)])
        start = np.concatenate([[0], np.cumsum(q_len)])
        out, _, mag, off = oracle.attention_batch_ref(qr, start, self.len, lambda s, h: (own[s][0][:, h], own[s][1][:, h]),
                                                      lambda h: (pre[0][:, h], pre[1][:, h]), D ** -0.5, H // KH)
        n = int(start[-1])
        got = synth.bf16_to_f32(host(b["out"]).view(np.uint16))
        keys = P + self.len.max()
        d = 2 * (D + 8) * 2.0 ** -24 * off + 2.0 ** -22 * (4 + keys / 32)
        tol = mag * (2 * d[..., None] + 2.0 ** -8 + (keys + 64) * 2.0 ** -24) + 2.0 ** -8 * np.abs(out) + 2.0 ** -133
        assert (np.abs(got - out)[:n] <= tol[:n]).all()
        want, a = oracle.gemv_ref(oracle.weights_exact(self.o_chunks, "q4_1", E, H * D), host(b["out"]).view(np.uint16).reshape(-1, H * D)[:n])
        assert oracle.tol_ratio(host(b["y"])[:n], want, a) <= 1.0


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_prompts_then_steps(kind):
    L = Layer(kind)
    L.prefix()
    prompts = [21, 1, 57]
    b = L.buffers(80, 57)
    L.fill(b, prompts)
    L.step(b)
    L.check_append(b, 79)
    L.check_attention(b, prompts)
    b = L.buffers(4, 1)
    for _ in range(4):
        L.fill(b, [1, 1, 1])
        L.step(b)
        L.check_append(b, 3)
        L.check_attention(b, [1, 1, 1])
    b = L.buffers(12, 4)                                # a window of drafted tokens, one sequence idle
    L.fill(b, [4, 0, 3])
    L.step(b)
    L.check_append(b, 7)
    L.check_attention(b, [4, 0, 3])


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_captured_steps(kind):
    """The same decode step eager and replayed, the tokens, slots and lengths changing between replays."""
    a, c = Layer(kind, "graph"), Layer(kind, "graph")
    bufs = []
    for L in (a, c):
        L.prefix()
        b = L.buffers(20, 9)
        L.fill(b, [9, 1, 8])
        L.step(b)
        bufs.append(L.buffers(3, 1))
    a.fill(bufs[0], [1, 1, 1])
    c.fill(bufs[1], [1, 1, 1])
    a.step(bufs[0])
    c.step(bufs[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step(bufs[1])
    for _ in range(5):
        a.fill(bufs[0], [1, 1, 1])
        c.fill(bufs[1], [1, 1, 1])
        a.step(bufs[0])
        graph.replay()
        torch.cuda.synchronize()
        for name in ("qr", "out", "y"):
            assert torch.equal(bufs[0][name], bufs[1][name])
        assert torch.equal(a.k, c.k) and torch.equal(a.v, c.v)


class Recurrent:
    """The mixer with states: q, k and v normalised to bf16, linear attention, the norm of its heads, the projection."""

    def __init__(self, M, n_seq, max_q, tag):
        g = self.g = synth.rng("gpu-mixing-linear", tag)
        self.M, self.n = M, n_seq
        rows = 3 * H * D
        self.w = weight(dev_u8(synth.gen_q4_1(g, rows, E, zero="normal")), rows, E, "q4_1")
        self.wo = weight(dev_u8(synth.gen_q4_1(g, E, H * D, zero="normal")), E, H * D, "q4_1")
        self.norm = dev_bf16(synth.bf16_bits(1 + 0.2 * g.standard_normal(D)))
        self.x = dev_bf16(synth.gen_x(g, M, E)).view(M, E)
        self.decay = dev_f32(-0.1 * g.random((M, H)))
        self.start, self.slots = torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda"), dev_i32(np.arange(n_seq))
        self.seqs = q().linear_attn_seqs(self.start, self.slots, max_q)
        self.state = dev_f32(g.standard_normal((n_seq, H, D, D)))
        self.qkv, self.b = torch.empty((M, rows), device="cuda"), torch.empty((M, rows), dtype=torch.int16, device="cuda")
        self.out, self.h, self.y = torch.empty((M, H, D), device="cuda"), torch.empty((M, H * D), dtype=torch.int16, device="cuda"), torch.empty((M, E), device="cuda")
        self.ws = torch.empty(q().linear_attn_ws(self.seqs, H, H, D, D, M), dtype=torch.uint8, device="cuda")
        self.gws = torch.zeros(max(256, q().gemm_block_ws(self.w), q().gemm_block_ws(self.wo)), dtype=torch.uint8, device="cuda")

    def step(self):
        M = self.M
        _gemm(self.w, self.x, self.qkv, M, self.gws)
        q().add_rmsnorm(self.qkv, self.norm, M * 3 * H, D, EPS, self.b)
        q().linear_attn(self.seqs, self.b[:, : H * D], self.b[:, H * D: 2 * H * D], self.b[:, 2 * H * D:], self.decay, H, H, D, D, M, D ** -0.5,
                        self.state, self.out, self.ws)
        q().add_rmsnorm(self.out, self.norm, M * H, D, EPS, self.h)
        _gemm(self.wo, self.h, self.y, M, self.gws)


@pytest.mark.parametrize("lens", [[1, 1, 1], [30, 1, 200]])
def test_recurrent_mixer(lens):
    """Three steps in a row, each from the state that the last one left; then the same captured."""
    M = sum(lens)
    r = Recurrent(M, 3, max(lens), "run")
    r.start.copy_(torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))
    states = [r.state.clone()]
    for _ in range(3):
        before = host(r.state).astype(np.float64)
        r.step()
        f = synth.bf16_to_f32(host(r.b).view(np.uint16)).reshape(M, 3, H, D)
        got, after, decay = host(r.out), host(r.state), host(r.decay)
        c = (5 * max(lens) + D + 96) * 2.0 ** -24
        at = 0
        for s, n in enumerate(lens):
            for h in range(H):
                out, S, mag, A = oracle.linear_attn_ref(f[at:at + n, 0, h], f[at:at + n, 1, h], f[at:at + n, 2, h], decay[at:at + n, h], D ** -0.5, before[s, h])
                assert (np.abs(got[at:at + n, h] - out) <= c * mag + 2.0 ** -130).all()
                assert (np.abs(after[s, h] - S) <= c * A + 2.0 ** -130).all()
            at += n
        states.append(r.state.clone())
    r.state.copy_(states[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.step()
    r.state.copy_(states[0])
    for want in states[1:]:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.state, want)


def test_steps_on_two_streams():
    rs = [Recurrent(3, 3, 1, f"stream{i}") for i in range(2)]
    want = []
    for r in rs:
        r.start.copy_(torch.tensor([0, 1, 2, 3], dtype=torch.int32))
        begin = r.state.clone()
        for _ in range(4):
            r.step()
        torch.cuda.synchronize()
        want.append((r.state.clone(), r.y.clone()))
        r.state.copy_(begin)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in rs]
    for _ in range(4):
        for r, s in zip(rs, streams):
            with torch.cuda.stream(s):
                r.step()
    torch.cuda.synchronize()
    for r, (state, y) in zip(rs, want):
        assert torch.equal(r.state, state) and torch.equal(r.y, y)
