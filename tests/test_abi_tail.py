"""Host-side refusals of q4nx_lora_add, q4nx_add_rmsnorm and q4nx_token_logprobs
(no call here reaches the device), also under the host sanitisers."""
import os
import subprocess
import sys

import pytest

from test_abi_host import LIB, _expect, q  # noqa: F401
from test_abi_sanitized import ROOT, _build_module

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")


def _table(q, **over):
    E, R, N, K = 4, 16, 64, 512
    args = dict(n_adapters=E, rank=R, rows=N, cols=K, a=0x100000, b=0x200000, scale=0x300000,
                a_bytes=E * R * K * 2, b_bytes=E * R * N * 2)
    args.update(over)
    return q.lora_table(**args)


WS = 0x10000000


def _add(q, L, **over):
    args = dict(x=0x400000, ids=0x500000, M=3, y=0x600000, ws=WS, base=None, stream=0, ws_bytes=1 << 24)
    args.update(over)
    q.lora_add(L, **args)


def test_lora_descriptor_rules(q):
    assert q.lora_ws(_table(q), 3) > 0
    for status, over in [
        (q.E_ARG, dict(a=0)), (q.E_ARG, dict(b=0)), (q.E_ARG, dict(scale=0)),
        (q.E_ARG, dict(n_adapters=0)), (q.E_ARG, dict(n_adapters=4097)),
        (q.E_SHAPE, dict(rank=0)), (q.E_SHAPE, dict(rank=12)), (q.E_SHAPE, dict(rank=264)),
        (q.E_SHAPE, dict(rows=48)), (q.E_SHAPE, dict(rows=0)), (q.E_SHAPE, dict(cols=300)),
        (q.E_SHAPE, dict(cols=(1 << 20) + 256)), (q.E_SHAPE, dict(rows=(1 << 20) + 32)),
        (q.E_SHAPE, dict(a_stride=16 * 512 * 2 - 16)), (q.E_SHAPE, dict(b_stride=0)),
        (q.E_SHAPE, dict(a_stride=-(16 * 512 * 2))), (q.E_SHAPE, dict(a_stride=2 ** 62, a_bytes=2 ** 63 - 1)),
        (q.E_SHORT, dict(a_bytes=4 * 16 * 512 * 2 - 1)), (q.E_SHORT, dict(b_bytes=4 * 16 * 64 * 2 - 1)),
        (q.E_SHORT, dict(a_stride=16 * 512 * 2 + 16)),
        (q.E_ALIGN, dict(a=0x100008)), (q.E_ALIGN, dict(b=0x200002)), (q.E_ALIGN, dict(a_stride=16 * 512 * 2 + 8)),
        (q.E_ALIGN, dict(scale=0x300002)), (q.E_ALIGN, dict(ranks=0x300001)),
    ]:
        _expect(q, status, _add, q, _table(q, **over))
        assert q.lora_ws(_table(q, **over), 3) == 0
    # padded strides are fine where the arena covers them
    assert q.lora_ws(_table(q, a_stride=16 * 512 * 2 + 16, a_bytes=3 * (16 * 512 * 2 + 16) + 16 * 512 * 2), 3) > 0


def test_lora_call_rules(q):
    L = _table(q)
    need = q.lora_ws(L, 3)
    y_bytes = 3 * 64 * 4
    for status, over in [
        (q.E_ARG, dict(M=0)), (q.E_ARG, dict(M=4097)), (q.E_ARG, dict(x=0)), (q.E_ARG, dict(ids=0)),
        (q.E_ARG, dict(y=0)), (q.E_ALIGN, dict(x=0x400008)), (q.E_ALIGN, dict(ids=0x500002)),
        (q.E_ALIGN, dict(y=0x600002)), (q.E_ALIGN, dict(base=0x700001)),
        (q.E_ARG, dict(base=0x600000 + y_bytes - 4)), (q.E_ARG, dict(base=0x600000 - y_bytes + 4)),
        (q.E_ARG, dict(y=0x400000 + 3 * 512 * 2 - 4)), (q.E_ARG, dict(y=0x500004)),
        (q.E_WORKSPACE, dict(ws=0)), (q.E_WORKSPACE, dict(ws_bytes=need - 1)), (q.E_ALIGN, dict(ws=WS + 16)),
    ]:
        _expect(q, status, _add, q, L, **over)
    assert q.lib().q4nx_lora_add(None, 0x1000, 0x2000, 1, 0x3000, 0x3000, WS, 1 << 20, None) == q.E_ARG
    assert q.lib().q4nx_lora_ws(None, 1) == 0 and q.lora_ws(L, 0) == 0 and q.lora_ws(L, 4097) == 0
    # a workspace grows with the rows, and the route's tables with the adapters
    assert q.lora_ws(L, 4096) > q.lora_ws(L, 300) > q.lora_ws(L, 1)


def test_lora_batched_rules(q):
    a, b = _table(q), _table(q, rank=8, rows=128, a_bytes=1 << 20, b_bytes=1 << 20)
    y1, y2, size = 0x600000, 0x700000, 3 * 64 * 4

    def call(jobs, **over):
        args = dict(x=0x400000, ids=0x500000, M=3, ws=WS, stream=0, ws_bytes=1)   # the workspace is checked last
        args.update(over)
        q.lora_add_batched(jobs, **args)
    _expect(q, q.E_WORKSPACE, call, [(a, None, y1), (b, None, y2)])
    assert q.lora_batched_ws([(a, None, y1), (b, None, y2)], 3) > q.lora_ws(a, 3)
    _expect(q, q.E_SHAPE, call, [(a, None, y1), (_table(q, cols=256), None, y2)])
    _expect(q, q.E_SHAPE, call, [(a, None, y1), (_table(q, n_adapters=3), None, y2)])
    _expect(q, q.E_SHAPE, call, [(a, None, y1), (_table(q, rank=9), None, y2)])
    assert "job 1" in q.last_error()
    _expect(q, q.E_ARG, call, [(a, None, y1), (b, None, y1 + size - 4)])     # y over y
    _expect(q, q.E_ARG, call, [(a, None, y1), (b, y1, y2)])                  # base of one over y of another
    _expect(q, q.E_WORKSPACE, call, [(a, 0x900000, y1), (b, 0x900000, y2)])  # a shared base is read only
    _expect(q, q.E_ARG, call, [(a, None, 0x600000 + 0x1000 * i) for i in range(9)])
    arr = (q.LoraJob * 1)()
    assert q.lib().q4nx_lora_add_batched(arr, 0, 0x1000, 0x2000, 1, WS, 1 << 20, None) == q.E_ARG
    assert q.lib().q4nx_lora_add_batched(None, 1, 0x1000, 0x2000, 1, WS, 1 << 20, None) == q.E_ARG
    assert q.lora_batched_ws([(a, None, y1), (_table(q, cols=256), None, y2)], 3) == 0


def test_lora_table_keeps_its_tensors(q):
    torch = pytest.importorskip("torch")
    a, b = torch.zeros(2, 8, 256, dtype=torch.bfloat16), torch.zeros(2, 32, 8, dtype=torch.bfloat16)
    s, y = torch.ones(2), torch.zeros(1, 32)
    L = q.lora_table(2, 8, 32, 256, a, b, s)
    assert L._owners[0] is a and L._owners[1] is b and L._owners[2] is s and q.lora_ws(L, 1) > 0
    assert q.lora_jobs([(L, None, y)])._owners[0][2] is y


def test_norm_rules(q):
    def call(**over):
        args = dict(r=0x200000, w=0x300000, M=4, D=300, eps=1e-6, x=0x400000, y=0x100000, r_out=0x500000, stream=0)
        args.update(over)
        q.add_rmsnorm(**args)
    f, h = 4 * 300 * 4, 4 * 300 * 2
    for status, over in [
        (q.E_ARG, dict(r=0)), (q.E_ARG, dict(w=0)), (q.E_ARG, dict(x=0)), (q.E_ARG, dict(M=0)),
        (q.E_ARG, dict(M=(1 << 20) + 1)), (q.E_SHAPE, dict(D=0)), (q.E_SHAPE, dict(D=32769)),
        (q.E_ARG, dict(eps=-1e-6)), (q.E_ARG, dict(eps=float("nan"))), (q.E_ARG, dict(eps=float("inf"))),
        (q.E_ALIGN, dict(y=0x100002)), (q.E_ALIGN, dict(r=0x200001)), (q.E_ALIGN, dict(r_out=0x500002)),
        (q.E_ALIGN, dict(w=0x300001)), (q.E_ALIGN, dict(x=0x400001)),
        (q.E_ARG, dict(x=0x200000)), (q.E_ARG, dict(x=0x100000 + f - 2)), (q.E_ARG, dict(x=0x500000 - h + 2)),
        (q.E_ARG, dict(x=0x300000 + 598)), (q.E_ARG, dict(r_out=0x200004)), (q.E_ARG, dict(r_out=0x100000 + f - 4)),
        (q.E_ARG, dict(r_out=0x300000 - f + 4)),
    ]:
        _expect(q, status, call, **over)


def test_logprobs_rules(q):
    def call(**over):
        args = dict(y=0x100000, n=5000, M=2, ws=WS, tokens=0x200000, n_tok=3, logp=0x300000, entropy=0x400000, k=4,
                    top_ids=0x500000, top_logp=0x600000, stream=0, ws_bytes=1 << 24)
        args.update(over)
        q.token_logprobs(**args)
    need = q.token_logprobs_ws(5000, 2, 4)
    assert need > q.token_logprobs_ws(5000, 2) > 0
    for bad in [(0, 1, 0), (10, 0, 0), (10, 65536, 0), ((1 << 20) + 1, 1, 0), (10, 1, -1), (100, 1, 33)]:
        assert q.token_logprobs_ws(*bad) == 0
    for status, over in [
        (q.E_ARG, dict(y=0)), (q.E_ARG, dict(n=0)), (q.E_ARG, dict(ldy=4999)), (q.E_ARG, dict(M=0)),
        (q.E_ARG, dict(M=65536)), (q.E_ARG, dict(n=(1 << 20) + 1)), (q.E_ARG, dict(n_tok=-1)),
        (q.E_ARG, dict(n_tok=65)), (q.E_ARG, dict(k=-1)), (q.E_ARG, dict(k=33)), (q.E_ARG, dict(n=3)),
        (q.E_ARG, dict(tokens=0)), (q.E_ARG, dict(logp=0)), (q.E_ARG, dict(top_ids=0)),
        (q.E_ARG, dict(n_tok=0, k=0, entropy=0)),
        (q.E_ALIGN, dict(y=0x100002)), (q.E_ALIGN, dict(tokens=0x200001)), (q.E_ALIGN, dict(logp=0x300002)),
        (q.E_ALIGN, dict(entropy=0x400001)), (q.E_ALIGN, dict(top_ids=0x500002)), (q.E_ALIGN, dict(top_logp=0x600003)),
        (q.E_WORKSPACE, dict(ws=0)), (q.E_WORKSPACE, dict(ws_bytes=need - 1)), (q.E_ALIGN, dict(ws=WS + 8)),
    ]:
        _expect(q, status, call, **over)


def test_refusals_are_clean_under_asan_and_ubsan():
    if os.environ.get("Q4NX_LIB"):
        pytest.skip("this is the sanitised run")
    b = _build_module()
    objs = [os.path.join(b.OBJDIR, s.replace(".hip", ".o")) for s in b.SOURCES if s != "api.hip"]
    rt = b.asan_runtime()
    if not all(os.path.exists(o) for o in objs) or not os.path.exists(rt):
        pytest.skip("the library's objects are not built, or no shared ASan runtime next to the compiler")
    lib = b.build_sanitized()
    pre = os.environ.get("LD_PRELOAD", "")
    env = dict(os.environ, LD_PRELOAD=rt + (":" + pre if pre else ""), Q4NX_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    here = os.path.abspath(__file__)
    r = subprocess.run([sys.executable, "-m", "pytest", here, "-q", "-p", "no:cacheprovider"], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "Sanitizer" not in out and "runtime error" not in out, out[-4000:]


@pytest.mark.parametrize("E", [1, 3, 40, 400])
@pytest.mark.parametrize("rank", [8, 64, 256])
@pytest.mark.parametrize("rows,cols", [(64, 256), (1 << 19, 256), (1 << 19, 4096), (2560, 9728), (4096, 14336), (64, 1 << 20)])
def test_a_workspace_for_many_rows_holds_fewer(q, E, rank, rows, cols):
    """A caller keeps one workspace for the largest batch, and a call past 2^31 bytes runs its pieces,
    the last of them shorter, in the one it was given."""
    L = q.Lora(E, rank, rows, cols, 4096, 4096, 2 * rank * cols, 2 * rank * rows, 1 << 60, 1 << 60, 4096, None)
    sizes = [q.lora_ws(L, M) for M in range(1, 4097)]
    assert sizes[0] > 0
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("n", [1, 700, 5000, 50001, 151936, 262144, 262145, 1 << 20])
@pytest.mark.parametrize("k", [0, 1, 32])
def test_a_logprobs_workspace_for_many_rows_holds_fewer(q, n, k):
    sizes = [q.token_logprobs_ws(n, M, min(k, n)) for M in [*range(1, 5000), 16383, 16384, 16385, 65535]]
    assert sizes[0] > 0
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_logprobs_outputs_lie_apart(q):
    """An output over the logits, the given tokens or another output is refused."""
    at = dict(y=0x1000000, tokens=0x2000000, logp=0x3000000, entropy=0x4000000, top_ids=0x5000000, top_logp=0x6000000)
    M, n, T, k = 4, 1000, 3, 5
    need = q.token_logprobs_ws(n, M, k)
    size = dict(y=((M - 1) * 1024 + n) * 4, tokens=M * T * 4, logp=M * T * 4, entropy=M * 4, top_ids=M * k * 4,
                top_logp=M * k * 4)
    for out in ("logp", "entropy", "top_ids", "top_logp"):
        for other in at:
            if other == out:
                continue
            for place in (at[other] + size[other] - 4, at[other] - size[out] + 4):
                args = dict(at, **{out: place})
                _expect(q, q.E_ARG, q.token_logprobs, n=n, M=M, ws=WS, n_tok=T, k=k, ldy=1024, stream=0, ws_bytes=need,
                        **args)


def test_lora_outputs_lie_apart_from_the_tables(q):
    """A y over an arena, the scales or the ranks, of its own job or another, is refused."""
    E, R, K = 4, 16, 512
    pad = 64

    def table(base, N):
        return q.lora_table(n_adapters=E, rank=R, rows=N, cols=K, a=base, b=base + 0x100000, scale=base + 0x200000,
                            ranks=base + 0x300000, a_stride=R * K * 2 + pad, b_stride=R * N * 2 + pad,
                            a_bytes=1 << 19, b_bytes=1 << 19)
    M, N = 3, 64
    size = M * N * 4
    t = [table(0x10000000 * (i + 2), N) for i in range(2)]
    parts = [(0, (E - 1) * (R * K * 2 + pad) + R * K * 2), (0x100000, (E - 1) * (R * N * 2 + pad) + R * N * 2),
             (0x200000, E * 4), (0x300000, E * 4)]
    apart = 0x600000

    def call(y0, y1=None, base=None):
        jobs = [(t[0], base, y0)] + ([(t[1], None, y1)] if y1 else [])
        q.lora_add_batched(jobs, 0x400000, 0x500000, M, WS, stream=0, ws_bytes=1)   # the workspace is checked last
    _expect(q, q.E_WORKSPACE, call, apart, apart + size)
    for at, n in parts:
        for table_at in (0x20000000, 0x30000000):
            lo = table_at + at
            for y in (lo - size + 4, lo, lo + n - 4):
                _expect(q, q.E_ARG, call, apart, y)
                _expect(q, q.E_ARG, call, y, apart)
                if table_at == 0x20000000:
                    _expect(q, q.E_ARG, call, y)
                    _expect(q, q.E_ARG, call, y, base=0x700000)
            for y in (lo - size, lo + n):
                _expect(q, q.E_WORKSPACE, call, apart, y)
    # a base over a table is read only
    _expect(q, q.E_WORKSPACE, call, apart, base=0x20000000)


def test_workspaces_lie_apart(q):
    """A workspace over an input or output is refused: where it begins in one, and where its last needed
    bytes reach one."""
    M, T, k, n = 4, 3, 5, 1000
    at = dict(y=0x1000000, tokens=0x2000000, logp=0x3000000, entropy=0x4000000, top_ids=0x5000000, top_logp=0x6000000)
    need = q.token_logprobs_ws(n, M, k)
    assert need % 256 == 0
    for name in at:
        for ws in (at[name], at[name] - need + 256):
            _expect(q, q.E_ARG, q.token_logprobs, n=n, M=M, ws=ws, n_tok=T, k=k, ldy=1024, stream=0, ws_bytes=1 << 22, **at)
            assert "workspace" in q.last_error()
    L = _table(q, ranks=0x800000)
    need = q.lora_ws(L, M)
    assert need % 256 == 0
    at = dict(a=0x100000, b=0x200000, scale=0x300000, ranks=0x800000, x=0x400000, ids=0x500000, y=0x600000, base=0x700000)
    for place in at.values():
        for ws in (place, place - need + 256):
            _expect(q, q.E_ARG, _add, q, L, M=M, base=at["base"], ws=ws, ws_bytes=1 << 22)
            assert "workspace" in q.last_error()


def test_logprobs_arrays_without_their_count(q):
    """Arrays that would be left unwritten without a word, because their count was left out, are refused;
    a count of 0 may stand beside them."""
    def call(**arrays):
        args = dict(entropy=0x400000, ws=WS, ws_bytes=1, stream=0)
        args.update(arrays)
        q.token_logprobs(0x100000, 5000, 2, **args)
    _expect(q, q.E_WORKSPACE, call)
    for arrays in (dict(tokens=0x200000, logp=0x300000), dict(tokens=0x200000), dict(logp=0x300000)):
        _expect(q, q.E_ARG, call, **arrays)
        _expect(q, q.E_ARG, call, k=3, top_ids=0x500000, **arrays)
        _expect(q, q.E_WORKSPACE, call, n_tok=0, **arrays)
    for arrays in (dict(top_ids=0x500000, top_logp=0x600000), dict(top_ids=0x500000), dict(top_logp=0x600000)):
        _expect(q, q.E_ARG, call, **arrays)
        _expect(q, q.E_WORKSPACE, call, k=0, **arrays)
    _expect(q, q.E_WORKSPACE, call, n_tok=1, tokens=0x200000, logp=0x300000, k=2, top_ids=0x500000)


def test_the_current_stream_by_either_way(q, monkeypatch):
    """Calls take the current stream of the current device, also with a torch that lacks the shorter way."""
    torch = pytest.importorskip("torch")

    class Stream:
        cuda_stream = 0x1234
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x1000 + device, raising=False)
    assert q._stream(None) == 0x1003
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert q._stream(None) == 0x1234
    assert q._stream(7) == 7 and q._stream(Stream) == 0x1234


@pytest.mark.parametrize("n", [1, 5, 31])
def test_no_more_alternatives_than_logits(q, n):
    """The workspace's size and the call agree on the largest k."""
    assert q.token_logprobs_ws(n, 3, n) > 0 and q.token_logprobs_ws(n, 3, n + 1) == 0
    args = dict(y=0x100000, n=n, M=3, ws=WS, ws_bytes=1, top_ids=0x500000, stream=0)
    _expect(q, q.E_WORKSPACE, q.token_logprobs, k=n, **args)
    _expect(q, q.E_ARG, q.token_logprobs, k=n + 1, **args)
