"""The tail of a step as it runs: a projection with adapters beside it, the
residual's norm, the head, and what is answered from its logits.

Each stage is checked against the float64 reference of its own inputs, which are
the device's outputs of the stage before; then the whole is captured in a graph
and replayed between eager work, and with several requests' steps on two streams.
"""
import numpy as np
import pytest

import oracle
import synth

from _gpu import dev_bf16, dev_f32, dev_i32, dev_u8, have_gpu, host, q, torch, weight

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

D, F, V, R, E, K_TOP = 512, 768, 4096, 16, 5, 6
EPS = 1e-6


class Step:
    """down projection [D, F] with adapters, final norm, Q8 head [V, D], log probabilities of M rows."""

    def __init__(self, M, tag):
        g = synth.rng("gpu-tail", tag, M)
        self.M = M
        self.down = synth.gen_q4_1(g, D, F, zero="normal")
        self.head = synth.gen_q8(g, V, D, "B")
        self.x = synth.gen_x(g, M, F)
        self.A = synth.bf16_bits(g.standard_normal((E, R, F)) / np.sqrt(F))
        self.B = synth.bf16_bits(g.standard_normal((E, D, R)))
        self.scale = np.linspace(0.5, 2, E).astype(np.float32)
        self.ids = g.integers(-1, E, M).astype(np.int32)
        self.r = g.standard_normal((M, D), dtype=np.float32)
        self.w = synth.bf16_bits(1 + 0.2 * g.standard_normal(D))
        self.tokens = g.integers(0, V, (M, 2)).astype(np.int32)
        f = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
        self.wd, self.wh = weight(dev_u8(self.down), D, F, "q4_1"), weight(dev_u8(self.head), V, D, "q8", "B")
        self.dx, self.dids, self.dr, self.dw = dev_bf16(self.x), dev_i32(self.ids), dev_f32(self.r), dev_bf16(self.w)
        self.table = q().lora_table(E, R, D, F, dev_bf16(self.A), dev_bf16(self.B), dev_f32(self.scale))
        self.dtok = dev_i32(self.tokens)
        self.y0, self.y, self.r_out, self.logits = f(M, D), f(M, D), f(M, D), f(M, V)
        self.h = torch.empty((M, D), dtype=torch.int16, device="cuda")
        self.lp, self.H, self.top = f(M, 2), f(M), f(M, K_TOP)
        self.top_ids = torch.empty((M, K_TOP), dtype=torch.int32, device="cuda")
        self.ws_gemm = torch.zeros(max(q().gemm_block_ws(self.wd), 256), dtype=torch.uint8, device="cuda")
        self.ws_lora = torch.empty(q().lora_ws(self.table, M), dtype=torch.uint8, device="cuda")
        self.ws_lp = torch.empty(q().token_logprobs_ws(V, M, K_TOP), dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        M = self.M
        if M <= q().GEMV_MAX_M:
            q().gemv(self.wd, self.dx, self.y0, M, stream=stream)
        else:
            q().gemm_block(self.wd, self.dx, self.y0, M, self.ws_gemm, stream=stream)
        q().lora_add(self.table, self.dx, self.dids, M, self.y, self.ws_lora, base=self.y0, stream=stream)
        q().add_rmsnorm(self.dr, self.dw, M, D, EPS, self.h, y=self.y, r_out=self.r_out, stream=stream)
        for m in range(0, M, q().GEMV_MAX_M):
            n = min(q().GEMV_MAX_M, M - m)
            q().gemv(self.wh, self.h[m:], self.logits[m:], n, stream=stream)
        q().token_logprobs(self.logits, V, M, self.ws_lp, tokens=self.dtok, n_tok=2, logp=self.lp, entropy=self.H,
                           k=K_TOP, top_ids=self.top_ids, top_logp=self.top, stream=stream)

    OUT = ("y0", "y", "r_out", "h", "logits", "lp", "H", "top_ids", "top")

    def outputs(self):
        return {n: host(getattr(self, n)).copy() for n in self.OUT}

    def clear(self):
        for n in self.OUT:
            getattr(self, n).zero_()


@pytest.mark.parametrize("M", [1, 4, 8, 40, 64])
def test_stage_by_stage(M):
    s = Step(M, "stage")
    s.run()
    o = s.outputs()
    want, a = oracle.gemv_ref(oracle.weights_exact(s.down, "q4_1", D, F), s.x)
    assert oracle.tol_ratio(o["y0"], want, a) <= 1.0
    # adapters: the bound of tests/test_gpu_lora.py
    want, mag = oracle.lora_ref(synth.bf16_to_f32(s.x), synth.bf16_to_f32(s.A), synth.bf16_to_f32(s.B), s.scale, s.ids, o["y0"])
    assert (np.abs(o["y"] - want) <= 2.0 ** -23 * ((F + 3 * R + 80) * mag + np.abs(o["y0"]) + np.abs(want))).all()
    np.testing.assert_array_equal(o["r_out"], o["y"] + s.r)
    _, want = oracle.add_rmsnorm_ref(None, o["r_out"], synth.bf16_to_f32(s.w), EPS)
    got = synth.bf16_to_f32(o["h"].view(np.uint16))
    assert (np.abs(got - want) <= (2.0 ** -8 + D * 2.0 ** -24) * np.abs(want) + 2.0 ** -134).all()
    want, a = oracle.gemv_ref(oracle.weights_exact(s.head, "q8", V, D, "B"), o["h"].view(np.uint16))
    assert oracle.tol_ratio(o["logits"], want, a) <= 1.0
    for m in range(0, M, 7):
        lp, H, ids, top, _ = oracle.token_logprobs_ref(o["logits"][m], s.tokens[m].tolist(), K_TOP)
        np.testing.assert_array_equal(o["top_ids"][m], ids)
        # 4096 terms: 64 additions a lane, a dozen joins, exponentials and logits of size < 64
        tol = 2.0 ** -23 * (120 + 3 * 64 + 2 * 64)
        np.testing.assert_allclose(np.concatenate([o["lp"][m], o["top"][m], o["H"][m:m + 1]]), lp + top + [H], atol=tol, rtol=0)
    # the head's own pick agrees with the first alternative
    idx = torch.empty(M, dtype=torch.int32, device="cuda")
    q().argmax(s.logits, V, M, idx)
    np.testing.assert_array_equal(host(idx), o["top_ids"][:, 0])


@pytest.mark.parametrize("M", [1, 8, 64])
def test_captured_and_replayed_between_eager_steps(M):
    s, t = Step(M, "graph"), Step(3, "beside")
    s.run()
    t.run()
    want, want_t = s.outputs(), t.outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(3):
        s.clear()
        t.clear()
        graph.replay()
        t.run()
        for n, v in s.outputs().items():
            np.testing.assert_array_equal(v, want[n], err_msg=n)
        for n, v in t.outputs().items():
            np.testing.assert_array_equal(v, want_t[n], err_msg=n)


def test_two_streams_with_workspaces_of_their_own():
    steps = [Step(8, "a"), Step(8, "b")]
    for s in steps:
        s.run()
    want = [s.outputs() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        s.clear()
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for n, v in s.outputs().items():
            np.testing.assert_array_equal(v, w[n], err_msg=n)


def test_two_graphs_share_workspaces():
    """Captured calls that share workspaces, replayed one after the other on one stream."""
    a, b = Step(8, "share-a"), Step(8, "share-b")
    b.ws_lora, b.ws_lp, b.ws_gemm = a.ws_lora, a.ws_lp, a.ws_gemm
    want = []
    graphs = []
    for s in (a, b):
        s.run()
        want.append(s.outputs())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for _ in range(3):
        a.clear()
        b.clear()
        for g in graphs + graphs[::-1]:
            g.replay()
        for s, w in zip((a, b), want):
            for n, v in s.outputs().items():
                np.testing.assert_array_equal(v, w[n], err_msg=n)


def test_routed_layer_after_the_norm():
    """The norm's output feeds the MoE router and experts as any bf16 activations do."""
    M, Dm, De, n_exp, k = 3, 512, 256, 8, 2
    g = synth.rng("gpu-tail", "moe")
    ex = {p: np.stack([synth.gen_q4_1(g, *((De, Dm) if p != "down" else (Dm, De)), zero="normal").reshape(-1)
                       for _ in range(n_exp)]) for p in ("gate", "up", "down")}
    gu, dn = ex["gate"].shape[1], ex["down"].shape[1]
    arenas = {p: dev_u8(v) for p, v in ex.items()}
    L = q().moe_layer(n_exp, Dm, De, "q4_1", arenas["gate"], arenas["up"], arenas["down"], gu, gu, dn)
    y, r = g.standard_normal((M, Dm), dtype=np.float32), g.standard_normal((M, Dm), dtype=np.float32)
    w, router = synth.bf16_bits(np.ones(Dm)), dev_bf16(synth.bf16_bits(g.standard_normal((n_exp, Dm)) / 20))
    x = torch.empty((M, Dm), dtype=torch.int16, device="cuda")
    ids, p = torch.empty((M, k), dtype=torch.int32, device="cuda"), torch.empty((M, k), device="cuda")
    z, Y = torch.empty((M, n_exp), device="cuda"), torch.empty((M, Dm), device="cuda")
    ws = torch.zeros(q().moe_ws(L, M, k), dtype=torch.uint8, device="cuda")
    q().add_rmsnorm(dev_f32(r), dev_bf16(w), M, Dm, EPS, x, y=dev_f32(y))
    q().moe_router(router, x, M, Dm, n_exp, k, ids, p, z)
    q().moe_experts(L, x, ids, p, Y, M, k, ws)

    def W(e):
        return tuple(oracle.weights_exact(ex[n][e].reshape(sh[0] // 32, sh[1] // 256, 5120), "q4_1", *sh)
                     for n, sh in (("gate", (De, Dm)), ("up", (De, Dm)), ("down", (Dm, De))))
    want, scale = oracle.moe_layer_ref(host(x).view(np.uint16), host(ids), host(p), W, None, n_experts=n_exp, with_scale=True)
    assert oracle.tol_ratio(host(Y), want, scale) <= 1.0
