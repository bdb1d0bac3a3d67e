"""Host-side refusals of q4nx_kv_append, q4nx_attention and q4nx_linear_attn (no call here reaches the
device), also under the host sanitisers."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_abi_host import LIB, q  # noqa: F401
from test_abi_sanitized import ROOT, _build_module

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

WS = 0x700000000000
KH, D, PAGE, PAGES = 2, 128, 16, 4
TOKENS = PAGES * PAGE * KH


def _expect(mod, status, fn, /, *a, **k):
    with pytest.raises(mod.Q4nxError) as e:
        fn(*a, **k)
    assert e.value.status == status, str(e.value)


def _cache(q, i8=False, **over):
    size = TOKENS * D * (1 if i8 else 2)
    args = dict(kv_heads=KH, head_dim=D, page_tokens=PAGE, n_pages=PAGES, k=0x1000000, v=0x2000000, k_bytes=size, v_bytes=size)
    if i8:
        args.update(k_scale=0x3000000, v_scale=0x4000000, k_scale_bytes=TOKENS * 4, v_scale_bytes=TOKENS * 4)
    args.update(over)
    return q.kv_cache(**args)


def _typed(q, kind):
    c = _cache(q)
    c.type = kind
    return c


def _cache_faults(q):
    """(status, cache) of every descriptor that each call refuses."""
    size = TOKENS * D * 2
    return [(s, _cache(q, **o)) for s, o in [
        (q.E_ARG, dict(kv_heads=0)), (q.E_ARG, dict(kv_heads=257)), (q.E_SHAPE, dict(head_dim=96)), (q.E_SHAPE, dict(head_dim=0)),
        (q.E_SHAPE, dict(head_dim=512)), (q.E_SHAPE, dict(page_tokens=8)), (q.E_SHAPE, dict(page_tokens=48)),
        (q.E_SHAPE, dict(page_tokens=2048)), (q.E_SHAPE, dict(page_tokens=0)), (q.E_ARG, dict(n_pages=0)),
        (q.E_ARG, dict(n_pages=2 ** 27)), (q.E_ARG, dict(n_pages=-1)), (q.E_ARG, dict(k=0)), (q.E_ARG, dict(v=0)),
        (q.E_ALIGN, dict(k=0x1000008)), (q.E_ALIGN, dict(v=0x2000002)), (q.E_SHORT, dict(k_bytes=size - 1)),
        (q.E_SHORT, dict(v_bytes=size - 1)), (q.E_ARG, dict(k_scale=0x3000000)), (q.E_ARG, dict(v_scale=0x3000000)),
    ]] + [(s, _cache(q, True, **o)) for s, o in [
        (q.E_ALIGN, dict(k_scale=0x3000004)), (q.E_ALIGN, dict(v_scale=0x4000008)), (q.E_SHORT, dict(k_scale_bytes=TOKENS * 4 - 1)),
        (q.E_SHORT, dict(v_scale_bytes=0)), (q.E_SHORT, dict(k_bytes=TOKENS * D - 1)), (q.E_ARG, dict(v_scale=0)),
    ]] + [(q.E_ARG, _typed(q, 2)), (q.E_ARG, _typed(q, -1))]


# ----------------------------------------------------------------------------
# kv_append
# ----------------------------------------------------------------------------
def _append(mod, cache=None, /, **over):
    args = dict(k=mod.heads(0x5000000, KH, D), v=mod.heads(0x6000000, KH, D), slots=0x7000000, M=3, rope=mod.rope(0x8000000, 0x8100000, D),
                q=mod.heads(0x9000000, 4, D), q_out=0xA000000, flags=0xB000000, stream=0)
    args.update(over)
    mod.kv_append(_cache(mod) if cache is None else cache, **args)


def test_append_rules(q):
    for status, cache in _cache_faults(q):
        _expect(q, status, _append, q, cache)
    h = lambda p, n, **k: q.heads(p, n, D, **k)  # noqa: E731
    for status, over in [
        (q.E_ARG, dict(M=0)), (q.E_ARG, dict(M=-1)), (q.E_ARG, dict(M=16385)), (q.E_ARG, dict(slots=0)), (q.E_ALIGN, dict(slots=0x7000002)),
        (q.E_ALIGN, dict(flags=0xB000001)), (q.E_ARG, dict(q_out=0)), (q.E_ARG, dict(q=None)), (q.E_ALIGN, dict(q_out=0xA000008)),
        (q.E_ARG, dict(k=h(0, KH))), (q.E_ARG, dict(v=h(0, KH))), (q.E_SHAPE, dict(k=h(0x5000000, 3))), (q.E_SHAPE, dict(v=h(0x6000000, 1))),
        (q.E_SHAPE, dict(k=h(0x5000000, KH, ld=KH * D - 1))), (q.E_SHAPE, dict(q=h(0x9000000, 4, ld=4 * D - 8))),
        (q.E_SHAPE, dict(q=h(0x9000000, 0))), (q.E_SHAPE, dict(q=h(0x9000000, 129))), (q.E_SHAPE, dict(q=h(0x9000000, 4, ld=2 ** 41))),
        (q.E_ALIGN, dict(k=h(0x5000002, KH))), (q.E_ALIGN, dict(k=h(0x5000001, KH, bf16=True))), (q.E_ALIGN, dict(q=h(0x9000001, 4))),
        (q.E_ARG, dict(rope=q.rope(0, 0x8100000, D))), (q.E_ARG, dict(rope=q.rope(0x8000000, 0, D))),
        (q.E_SHAPE, dict(rope=q.rope(0x8000000, 0x8100000, 0))), (q.E_SHAPE, dict(rope=q.rope(0x8000000, 0x8100000, 8))),
        (q.E_SHAPE, dict(rope=q.rope(0x8000000, 0x8100000, 144))), (q.E_SHAPE, dict(rope=q.rope(0x8000000, 0x8100000, 40))),
        (q.E_ALIGN, dict(rope=q.rope(0x8000002, 0x8100000, D))), (q.E_ALIGN, dict(rope=q.rope(0x8000000, 0x8100001, D))),
    ]:
        _expect(q, status, _append, q, **over)
    bad = q.heads(0x5000000, KH, D)
    bad.type = 2
    _expect(q, q.E_ARG, _append, q, k=bad)
    lib, null = q.lib().q4nx_kv_append, None
    assert lib(null, null, null, 0, null, null, 0x7000000, 1, 0, None) == q.E_ARG
    assert lib(ctypes.byref(_cache(q)), null, null, 0, null, null, 0x7000000, 1, 0, None) == q.E_ARG


def test_append_outputs_apart(q):
    """q_out, the cache and the flags lie apart from the inputs and each other, up to the last byte."""
    kb, qb, cb = 3 * KH * D * 4, 3 * 4 * D * 2, TOKENS * D * 2
    for over in [dict(q_out=0x5000000), dict(q_out=0x5000000 + kb - 16), dict(q_out=0x1000000 + cb - 16), dict(q_out=0x2000000 - qb + 16),
                 dict(q_out=0x7000000), dict(q_out=0x8000000), dict(q_out=0x8100000), dict(q_out=0x9000000), dict(q_out=0xB000000),
                 dict(k=q.heads(0x1000000 + cb - 4, KH, D)), dict(v=q.heads(0x2000000, KH, D)), dict(slots=0x1000000),
                 dict(slots=0x2000000 + cb - 4), dict(flags=0x7000008), dict(flags=0x1000000), dict(rope=q.rope(0x1000000, 0x8100000, D)),
                 dict(q=q.heads(0x2000000 + 4, 4, D))]:
        _expect(q, q.E_ARG, _append, q, **over)
    _expect(q, q.E_ARG, _append, q, _cache(q, v=0x1000000))
    _expect(q, q.E_ARG, _append, q, _cache(q, True, v_scale=0x3000000))
    _expect(q, q.E_ARG, _append, q, _cache(q, True, k_scale=0x1000000))


def test_append_binding(q):
    torch = pytest.importorskip("torch")
    c = _cache(q)
    k = torch.zeros(3, KH * D)
    for bad in (torch.zeros(3, KH * D, dtype=torch.float64), torch.zeros(3, KH * D, dtype=torch.int8)):
        _expect(q, q.E_ARG, q.kv_append, c, bad, k, 0x7000000, 3, stream=0)
    _expect(q, q.E_SHAPE, q.kv_append, c, torch.zeros(KH * D, 3).t(), k, 0x7000000, 3, stream=0)
    _expect(q, q.E_SHAPE, q.kv_append, c, torch.zeros(3, KH, 2 * D)[:, :, :D], k, 0x7000000, 3, stream=0)
    _expect(q, q.E_ARG, q.kv_append, c, k, k, 0x7000000, 3, q=k, stream=0)               # q without q_heads
    wide = torch.zeros(3, 10 * D)
    h = q.heads(wide[:, D:3 * D], KH, D)
    assert (h.ld, h.type, h.heads) == (10 * D, 0, KH)
    h = q.heads(torch.zeros(1, KH, D, dtype=torch.bfloat16), KH, D)
    assert (h.ld, h.type) == (KH * D, 1)
    assert q.heads(wide[:1, D:3 * D], KH, D).ld == 10 * D and q.heads(wide.view(-1), KH, D).ld == KH * D


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------
def _batch(q, **over):
    args = dict(q_start=0x5000000, kv_len=0x5100000, pages=0x5200000, max_q=1, n_seq=3, pages_ld=2, prefix_len=20, prefix_pages=0x5300000)
    args.update(over)
    return q.attn_batch(**args)


def _attend(mod, cache=None, batch=None, /, **over):
    args = dict(q=0x6000000, q_heads=4, M=3, scale=0.1, out=0x7000000, ws=WS, lse=0x8000000, flags=0x9000000, stream=0, ws_bytes=1 << 40)
    args.update(over)
    mod.attention(_cache(mod) if cache is None else cache, _batch(mod) if batch is None else batch, **args)


def test_attention_rules(q):
    for status, cache in _cache_faults(q):
        _expect(q, status, _attend, q, cache)
    for status, over in [(q.E_ARG, dict(n_seq=0)), (q.E_ARG, dict(n_seq=1025)), (q.E_ARG, dict(max_q=0)), (q.E_ARG, dict(max_q=65537)),
                         (q.E_ARG, dict(q_start=0)), (q.E_ARG, dict(kv_len=0)), (q.E_ARG, dict(pages=0)), (q.E_ARG, dict(prefix_pages=0)),
                         (q.E_ARG, dict(pages_ld=0)), (q.E_ARG, dict(prefix_len=-1)), (q.E_ARG, dict(prefix_len=2 ** 31 - 1)),
                         (q.E_ARG, dict(pages_ld=2 ** 27)), (q.E_ALIGN, dict(q_start=0x5000002)), (q.E_ALIGN, dict(kv_len=0x5100001)),
                         (q.E_ALIGN, dict(pages=0x5200002)), (q.E_ALIGN, dict(prefix_pages=0x5300002))]:
        _expect(q, status, _attend, q, None, _batch(q, **over))
    for status, over in [(q.E_ARG, dict(M=0)), (q.E_ARG, dict(M=65537)), (q.E_SHAPE, dict(q_heads=0)), (q.E_SHAPE, dict(q_heads=3)),
                         (q.E_SHAPE, dict(q_heads=130)), (q.E_ARG, dict(scale=float("inf"))), (q.E_ARG, dict(scale=float("nan"))),
                         (q.E_ARG, dict(q=0)), (q.E_ARG, dict(out=0)), (q.E_ALIGN, dict(q=0x6000008)), (q.E_ALIGN, dict(out=0x7000004)),
                         (q.E_ALIGN, dict(lse=0x8000002)), (q.E_ALIGN, dict(flags=0x9000002)), (q.E_WORKSPACE, dict(ws=0)),
                         (q.E_ALIGN, dict(ws=WS + 64))]:
        _expect(q, status, _attend, q, **over)
    lib = q.lib().q4nx_attention
    assert lib(None, ctypes.byref(_batch(q)), 0x6000000, 4, 3, 0.1, 0x7000000, 0, WS, 1 << 40, 0, None) == q.E_ARG
    assert lib(ctypes.byref(_cache(q)), None, 0x6000000, 4, 3, 0.1, 0x7000000, 0, WS, 1 << 40, 0, None) == q.E_ARG


@pytest.mark.parametrize("q_heads,max_q,prefix", [(4, 1, 0), (4, 1, 20), (4, 12, 20), (32, 2, 3), (2, 5000, 20), (2, 5000, 0)])
def test_attention_workspace(q, q_heads, max_q, prefix):
    """The size's function and the call agree, whichever kernels the shape takes."""
    c, b = _cache(q), _batch(q, max_q=max_q, prefix_len=prefix)
    for M in (1, 3, 64, 5000):
        need = q.attention_ws(c, b, q_heads, M)
        assert need > 0 and need % 256 == 0
        _expect(q, q.E_WORKSPACE, _attend, q, c, b, q_heads=q_heads, M=M, ws_bytes=need - 1)
    assert q.attention_ws(c, b, q_heads, 0) == 0 and q.attention_ws(c, b, 3, 1) == 0
    assert q.attention_ws(_cache(q, head_dim=96), b, q_heads, 1) == 0
    assert q.attention_ws(_cache(q, k=0, v=0), b, q_heads, 1) > 0      # pointers are not looked at


@pytest.mark.parametrize("max_q", [1, 4, 9, 16, 100])
@pytest.mark.parametrize("prefix", [0, 20])
@pytest.mark.parametrize("q_heads", [2, 4, 32])
def test_attention_workspace_grows_with_the_rows(q, max_q, prefix, q_heads):
    need = [q.attention_ws(_cache(q), _batch(q, max_q=max_q, prefix_len=prefix), q_heads, M) for M in [*range(1, 300), 4096, 65536]]
    assert need == sorted(need)


def test_attention_outputs_apart(q):
    c, b = _cache(q), _batch(q)
    need, size, cb = q.attention_ws(c, b, 4, 3), 3 * 4 * D * 2, TOKENS * D * 2
    for over in [dict(out=0x6000000), dict(out=0x6000000 + size - 16), dict(out=0x1000000 + cb - 16), dict(out=0x2000000), dict(out=0x5000000),
                 dict(out=0x8000000), dict(out=0x9000000), dict(lse=0x6000000), dict(lse=0x7000000 + size - 4), dict(lse=0x5100000),
                 dict(lse=0x5200000 + 20), dict(lse=0x5300000 + 4), dict(flags=0x5000000 + 12), dict(flags=0x8000000), dict(flags=0x2000000),
                 dict(out=WS), dict(lse=WS + need - 4), dict(flags=WS), dict(q=WS + need - 16)]:
        _expect(q, q.E_ARG, _attend, q, c, b, **over)
    _expect(q, q.E_ARG, _attend, q, c, _batch(q, pages=WS + need - 4))
    _expect(q, q.E_ARG, _attend, q, _cache(q, True, v_scale=0x7000000), b)
    _expect(q, q.E_ARG, _attend, q, _cache(q, k=WS), b)


# ----------------------------------------------------------------------------
# linear attention
# ----------------------------------------------------------------------------
def _linear(mod, seqs=None, /, **over):
    args = dict(q=0x1000000, k=0x2000000, v=0x3000000, decay=0x4000000, k_heads=2, v_heads=4, dk=64, dv=128, M=3, scale=0.5, state=0x5000000,
                out=0x7000000, ws=WS, state_out=0x6000000, flags=0x8000000, stream=0, n_slots=3, ws_bytes=1 << 40)
    args.update(over)
    mod.linear_attn(_seqs(mod) if seqs is None else seqs, **args)


def _seqs(q, **over):
    args = dict(q_start=0x9000000, slots=0x9100000, max_q=1, fresh=0x9200000, n_seq=2)
    args.update(over)
    return q.linear_attn_seqs(**args)


def test_linear_rules(q):
    for status, over in [(q.E_ARG, dict(n_seq=0)), (q.E_ARG, dict(n_seq=1025)), (q.E_ARG, dict(max_q=0)), (q.E_ARG, dict(max_q=65537)),
                         (q.E_ARG, dict(q_start=0)), (q.E_ARG, dict(slots=0)), (q.E_ALIGN, dict(q_start=0x9000001)),
                         (q.E_ALIGN, dict(slots=0x9100002)), (q.E_ALIGN, dict(fresh=0x9200002))]:
        _expect(q, status, _linear, q, _seqs(q, **over))
    for status, over in [(q.E_ARG, dict(M=0)), (q.E_ARG, dict(M=65537)), (q.E_ARG, dict(n_slots=0)), (q.E_ARG, dict(n_slots=(1 << 20) + 1)),
                         (q.E_SHAPE, dict(k_heads=0)), (q.E_SHAPE, dict(k_heads=3)), (q.E_SHAPE, dict(v_heads=5)), (q.E_SHAPE, dict(v_heads=1026)),
                         (q.E_SHAPE, dict(k_heads=257, v_heads=257)), (q.E_SHAPE, dict(dk=96)), (q.E_SHAPE, dict(dv=256)), (q.E_SHAPE, dict(dv=0)),
                         (q.E_SHAPE, dict(q_ld=120)), (q.E_SHAPE, dict(k_ld=0)), (q.E_SHAPE, dict(v_ld=504)), (q.E_SHAPE, dict(decay_ld=3)),
                         (q.E_SHAPE, dict(decay_ld=-4)), (q.E_SHAPE, dict(q_ld=(1 << 24) + 8)), (q.E_SHAPE, dict(v_ld=-512)),
                         (q.E_ALIGN, dict(q_ld=132)), (q.E_ALIGN, dict(k_ld=129)), (q.E_ALIGN, dict(v_ld=516)),
                         (q.E_ARG, dict(scale=float("nan"))), (q.E_ARG, dict(scale=-float("inf"))), (q.E_ALIGN, dict(q=0x1000008)),
                         (q.E_ALIGN, dict(k=0x2000002)), (q.E_ALIGN, dict(v=0x3000004)), (q.E_ALIGN, dict(decay=0x4000002)),
                         (q.E_ALIGN, dict(state=0x5000004)), (q.E_ALIGN, dict(state_out=0x6000008)), (q.E_ALIGN, dict(out=0x7000004)),
                         (q.E_ALIGN, dict(flags=0x8000002)), (q.E_WORKSPACE, dict(ws=0)), (q.E_ALIGN, dict(ws=WS + 16))]:
        _expect(q, status, _linear, q, **over)
    for name in ("q", "k", "v", "decay", "state", "out"):
        _expect(q, q.E_ARG, _linear, q, **{name: 0})
    _expect(q, q.E_ARG, _linear, q, state_out=0)
    assert q.lib().q4nx_linear_attn(None, 1, 1, 1, 1, 1, 1, 1, 0, 1, 0.5, 1, 1, 1, WS, 1 << 40, 0, None) == q.E_ARG
    assert q.lib().q4nx_linear_attn_ws(None, 1) == 0


@pytest.mark.parametrize("max_q", [1, 13, 200, 60000])
def test_linear_workspace(q, max_q):
    s = _seqs(q, max_q=max_q)
    for M in (1, 65, 4096, 65536):
        need = q.linear_attn_ws(s, 2, 4, 64, 128, M)
        assert need > 0 and need % 256 == 0
        _expect(q, q.E_WORKSPACE, _linear, q, s, M=M, ws_bytes=need - 1, q=0x100000000, k=0x200000000, v=0x300000000, decay=0x400000000,
                out=0x500000000)
    assert q.linear_attn_ws(s, 2, 5, 64, 128, 1) == 0 and q.linear_attn_ws(s, 2, 4, 64, 96, 1) == 0 and q.linear_attn_ws(s, 2, 4, 64, 128, 0) == 0


def test_linear_outputs_apart(q):
    sb, ob, need = 3 * 4 * 64 * 128 * 4, 3 * 4 * 128 * 4, 256
    for over in [dict(state_out=0x5000010), dict(state_out=0x5000000 + sb - 16), dict(state_out=0x5000000 - sb + 16), dict(out=0x5000000 + sb - 16),
                 dict(out=0x6000000), dict(out=0x1000000), dict(out=0x2000000), dict(out=0x3000000), dict(out=0x4000000), dict(out=0x9000000),
                 dict(out=0x9100000), dict(out=0x9200000), dict(out=0x7000000, flags=0x7000000 + ob - 4), dict(flags=0x9000000),
                 dict(flags=0x6000000), dict(out=WS), dict(state_out=WS), dict(state=WS + need - 16), dict(q=WS), dict(decay=WS)]:
        _expect(q, q.E_ARG, _linear, q, **over)


def test_linear_binding(q):
    torch = pytest.importorskip("torch")
    _expect(q, q.E_SHAPE, _linear, q, q=torch.zeros(128, 3, dtype=torch.bfloat16).t())
    _expect(q, q.E_SHAPE, _linear, q, v=torch.zeros(3, 4, 256, dtype=torch.bfloat16)[:, :, :128])
    _expect(q, q.E_SHAPE, _linear, q, decay=torch.zeros(4, 3).t())


def test_types_and_dimensions_that_are_not_taken(q):
    torch = pytest.importorskip("torch")
    c, k = _cache(q), torch.zeros(3, KH * D)
    for dtype in (torch.float16, torch.int32, torch.uint8):
        _expect(q, q.E_ARG, q.kv_append, c, k.to(dtype), k, 0x7000000, 3, stream=0)
        _expect(q, q.E_ARG, q.kv_append, c, k, k.to(dtype), 0x7000000, 3, stream=0)
        _expect(q, q.E_ARG, q.heads, k.to(dtype), KH, D)
    assert q.heads(torch.zeros(3, KH * D, dtype=torch.int16), KH, D).type == 1
    _expect(q, q.E_SHAPE, q.kv_append, c, torch.zeros(1, 3, KH, D), k, 0x7000000, 3, stream=0)
    for scale in (3e38, -2.5e38, float("nan")):      # times log2(e) beyond fp32
        _expect(q, q.E_ARG, _attend, q, scale=scale)


def test_linear_sequences_may_change_between_calls(q):
    s = _seqs(q, max_q=1)
    few = q.linear_attn_ws(s, 2, 4, 64, 128, 4096)
    s.max_q = 4096
    long = q.linear_attn_ws(s, 2, 4, 64, 128, 4096)
    assert few == q.linear_attn_ws(_seqs(q, max_q=1), 2, 4, 64, 128, 4096) < long == q.linear_attn_ws(_seqs(q, max_q=4096), 2, 4, 64, 128, 4096)
    _expect(q, q.E_WORKSPACE, _linear, q, s, M=4096, ws_bytes=long - 1, q=0x100000000, k=0x200000000, v=0x300000000, decay=0x400000000,
            out=0x500000000)
    assert (s.k_heads, s.v_heads, s.n_slots) == (0, 0, 0)


def test_page_tables_that_are_strided_binding(q):
    """A table's rows are as far apart as its strides say; what cannot be said so is refused."""
    torch = pytest.importorskip("torch")
    wide, lens = torch.arange(60, dtype=torch.int32).view(4, 15), torch.ones(4, dtype=torch.int32)
    start = torch.arange(5, dtype=torch.int32)
    b = q.attn_batch(start, lens, wide[:, :6], 1)
    assert (b.pages, b.pages_ld, b.n_seq) == (wide.data_ptr(), 15, 4)
    assert q.attn_batch(start, lens, wide, 1).pages_ld == 15
    assert q.attn_batch(start, lens[::2][:2].contiguous(), wide[::2, :6], 1).pages_ld == 30
    assert q.attn_batch(start[:4], lens[:3], wide[:3, 4:9], 1).pages_ld == 15       # the fourth row is there behind them
    assert q.attn_batch(start[:2], lens[:1], wide[:1, 4:9], 1).pages_ld == 5        # one row: its own columns
    assert q.attn_batch(start, lens, wide[:, :6], 1, pages_ld=15).pages_ld == 15
    for bad in (wide.t(), wide[:, ::2], wide[:1].expand(4, 15), wide[:, 4:9], wide[0], wide.view(2, 2, 15)):
        _expect(q, q.E_SHAPE, q.attn_batch, start, lens, bad, 1)


def test_arrays_in_one_piece_binding(q):
    """A strided tensor is refused where the call takes no stride: it would be read or written at other places."""
    torch = pytest.importorskip("torch")
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    z = lambda *s, t=f32: torch.zeros(*s, dtype=t)  # noqa: E731
    shape = (PAGES, KH, PAGE * D)
    for over in (dict(k=z(PAGES, 2, KH, PAGE * D, t=bf)[:, 0]), dict(v=z(*shape[:2], 2 * PAGE * D, t=bf)[..., ::2])):
        _expect(q, q.E_SHAPE, _cache, q, **over)
    for name in ("k_scale", "v_scale"):
        _expect(q, q.E_SHAPE, _cache, q, True, **{name: z(PAGES, PAGE, KH).transpose(1, 2)})
    _expect(q, q.E_SHAPE, q.rope, z(2 * D)[::2], 0x8100000, D)
    _expect(q, q.E_SHAPE, q.rope, 0x8000000, z(6, t=i32)[::2], D)
    _expect(q, q.E_SHAPE, _append, q, slots=z(3, 2, t=i32)[:, 0])
    _expect(q, q.E_SHAPE, _append, q, q_out=z(3, 8, D, t=bf)[:, :4])
    for name, bad in (("k", z(2 * KH * D)[::2]), ("v", z(2 * KH * D, t=bf)[::2]), ("q", z(8 * D)[::2])):
        _expect(q, q.E_SHAPE, _append, q, M=1, q_heads=4, **{name: bad})
    for over in (dict(q_start=z(8, t=i32)[::2]), dict(kv_len=z(6, t=i32)[::2]), dict(prefix_pages=z(2, 2, t=i32)[:, 1])):
        _expect(q, q.E_SHAPE, _batch, q, **over)
    for over in (dict(q=z(3, 8, D, t=bf)[:, :4]), dict(out=z(4, 3, D, t=bf).transpose(0, 1)), dict(lse=z(4, 3).t())):
        _expect(q, q.E_SHAPE, _attend, q, **over)
    for over in (dict(q_start=z(6, t=i32)[::2]), dict(slots=z(2, 2, t=i32)[:, 0]), dict(fresh=z(4, t=i32)[::2])):
        _expect(q, q.E_SHAPE, _seqs, q, **over)
    for over in (dict(state=z(3, 4, 128, 64).transpose(2, 3)), dict(state_out=z(3, 8, 64, 128)[:, :4]), dict(out=z(3, 4, 256)[..., :128]),
                 dict(decay=z(4, 2)[:, 0]), dict(q=z(256, t=bf)[::2])):
        _expect(q, q.E_SHAPE, _linear, q, **over)


def test_indexes_of_another_type_binding(q):
    """Slots, positions, starts, lengths and pages of a wider type are refused: its halves would be taken for indexes."""
    torch = pytest.importorskip("torch")
    for t in (torch.int64, torch.int16, torch.float32, torch.bool):
        z = lambda *s: torch.zeros(*s, dtype=t)  # noqa: B023, E731
        _expect(q, q.E_ARG, _append, q, slots=z(3))
        _expect(q, q.E_ARG, q.rope, 0x8000000, z(3), D)
        for over in (dict(q_start=z(4)), dict(kv_len=z(3)), dict(prefix_pages=z(2)), dict(pages=z(3, 2), pages_ld=None)):
            _expect(q, q.E_ARG, _batch, q, **over)
        for over in (dict(q_start=z(3)), dict(slots=z(2)), dict(fresh=z(2))):
            _expect(q, q.E_ARG, _seqs, q, **over)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    b = q.attn_batch(z(4), z(3), z(3, 2), 1, prefix_len=5, prefix_pages=z(1))
    assert (b.n_seq, b.pages_ld) == (3, 2) and q.linear_attn_seqs(z(4), z(3), 1, fresh=z(3)).n_seq == 3


@pytest.mark.parametrize("max_q", [12, 100, 193, 1000, 65536])
@pytest.mark.parametrize("k_heads,v_heads,n_seq", [(1, 1, 1), (2, 4, 3), (16, 32, 1), (16, 32, 7), (100, 200, 1), (16, 128, 2), (1, 1, 255)])
def test_linear_workspace_grows_with_the_rows(q, max_q, k_heads, v_heads, n_seq):
    s = _seqs(q, max_q=max_q, n_seq=n_seq)
    need = [q.linear_attn_ws(s, k_heads, v_heads, 64, 128, M) for M in [*range(1, 4000), 4096, 8192, 8193, 20000, 65535, 65536]]
    assert min(need) > 0 and need == sorted(need)


def test_one_column_at_any_stride_binding(q):
    """The decays of a single head may be a column of a transposed array: the step between rows is all that counts."""
    torch = pytest.importorskip("torch")
    for decay in (torch.zeros(1, 3).t(), torch.zeros(2, 3).t()[:, :1], torch.zeros(3, 5)[:, 2:3]):
        _expect(q, q.E_WORKSPACE, _linear, q, k_heads=1, v_heads=1, decay=decay, ws=0)       # past the strides' checks
    _expect(q, q.E_SHAPE, _linear, q, k_heads=1, v_heads=2, decay=torch.zeros(2, 3).t())


# ----------------------------------------------------------------------------
# the checks under the host sanitisers
# ----------------------------------------------------------------------------
def test_mixing_checks_are_clean_under_asan_and_ubsan():
    b = _build_module()
    objs = [os.path.join(b.OBJDIR, s.replace(".hip", ".o")) for s in b.SOURCES if s != "api.hip"]
    if os.environ.get("Q4NX_LIB") or not all(os.path.exists(o) for o in objs):
        pytest.skip("the library's objects are not built, or this is the sanitised run")
    rt = b.asan_runtime()
    if not os.path.exists(rt):
        pytest.skip("no shared ASan runtime next to the compiler")
    lib = b.build_sanitized()
    pre = os.environ.get("LD_PRELOAD", "")
    env = dict(os.environ, LD_PRELOAD=rt + (":" + pre if pre else ""), Q4NX_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    child = (
        "import sys, pytest\n"
        f"rc = pytest.main([{os.path.join(ROOT, 'tests', 'test_abi_mixing.py')!r}, '-q', '-p', 'no:cacheprovider', '-k', 'not binding'])\n"
        "maps = open('/proc/self/maps').read()\n"
        f"print('sanitised library loaded:', {lib!r} in maps and 'libclang_rt.asan' in maps)\n"
        "sys.exit(int(rc))\n")
    r = subprocess.run([sys.executable, "-c", child], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "Sanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert "sanitised library loaded: True" in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
