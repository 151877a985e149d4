"""Refusals of the ragged products, the integer products and the route grouping,
on the host: nothing here launches GPU work."""
import ctypes as C

import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from block_scaled_fp4_histogram_amd import _lib

P = 4096   # an aligned address that is never read


def _mm(L, **kw):
    a = dict(dtype=M.T_BF16, x=P, x_rows=64, rows=None, w=P, first=P, E=4, R=64, N=64, K=64, out_dtype=M.T_BF16, out=P)
    a.update(kw)
    return L.moe_grouped_mm(a["dtype"], a["x"], a["x_rows"], a["rows"], a["w"], a["first"], a["E"], a["R"], a["N"],
                            a["K"], a["out_dtype"], a["out"], None, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=M.T_FP32), M.MOE_EUNSUPPORTED), (dict(dtype=9), M.MOE_EUNSUPPORTED),
    (dict(out_dtype=M.T_FP16), M.MOE_EUNSUPPORTED), (dict(N=60), M.MOE_EUNSUPPORTED), (dict(K=65), M.MOE_EUNSUPPORTED),
    (dict(N=0), M.MOE_EINVAL), (dict(K=-8), M.MOE_EINVAL), (dict(R=-1), M.MOE_EINVAL), (dict(E=0), M.MOE_EINVAL),
    (dict(E=1025), M.MOE_EUNSUPPORTED), (dict(K=(1 << 20) + 8), M.MOE_EUNSUPPORTED), (dict(x=None), M.MOE_EINVAL),
    (dict(w=P + 8), M.MOE_EINVAL), (dict(out=P + 2), M.MOE_EINVAL), (dict(first=None), M.MOE_EINVAL),
    (dict(first=P + 2), M.MOE_EINVAL), (dict(rows=P + 1), M.MOE_EINVAL), (dict(x_rows=63), M.MOE_EINVAL),
    (dict(x_rows=-1, rows=P), M.MOE_EINVAL), (dict(R=0), M.MOE_OK), (dict(R=0, x=None, out=None), M.MOE_OK)])
def test_forward_refusals(kw, code):
    L = _lib.load()
    assert _mm(L, **kw) == code
    if code != M.MOE_OK:
        assert L.moe_last_error().decode().startswith("moe_grouped_mm")


def test_gradient_refusals():
    L = _lib.load()
    assert L.moe_grouped_mm_dx(M.T_BF16, P, P, P, 4, 64, 12, 64, M.T_BF16, P, None, 0, None) == M.MOE_EUNSUPPORTED
    assert L.moe_grouped_mm_dx(M.T_BF16, None, P, P, 4, 64, 16, 64, M.T_BF16, P, None, 0, None) == M.MOE_EINVAL
    assert L.moe_grouped_mm_dx(M.T_BF16, P, P, P, 4, 0, 16, 64, M.T_BF16, P, None, 0, None) == M.MOE_OK
    dw = lambda od, acc, x=P, out=P: L.moe_grouped_mm_dw(M.T_FP16, P, x, 64, None, P, 4, 64, 16, 64, od, acc, out, None, 0, None)  # noqa: E731
    assert dw(M.T_FP16, 1) == M.MOE_EUNSUPPORTED and b"accumulate" in L.moe_last_error()
    assert dw(M.T_BF16, 0) == M.MOE_EUNSUPPORTED
    assert dw(M.T_FP32, 0, x=None) == M.MOE_EINVAL
    assert dw(M.T_FP32, 0, out=P + 4) == M.MOE_EINVAL


def test_int8_refusals():
    L = _lib.load()
    q = lambda dt, r, c, x=P, o=P, s=P: L.moe_quant_int8(dt, x, r, c, o, s, None)  # noqa: E731
    assert q(M.T_FP32, 4, 64) == M.MOE_EUNSUPPORTED and q(M.T_BF16, 4, 24) == M.MOE_EUNSUPPORTED
    assert q(M.T_BF16, -1, 64) == M.MOE_EINVAL and q(M.T_BF16, 4, 64, x=P + 4) == M.MOE_EINVAL
    assert q(M.T_BF16, 4, 64, s=None) == M.MOE_EINVAL and q(M.T_BF16, 0, 64) == M.MOE_OK
    mm = lambda m, n, k, od, xs=P, x=P: L.moe_int8_mm(x, xs, P, P, m, n, k, od, P, None, 0, None)  # noqa: E731
    assert mm(4, 8, 24, M.T_BF16) == M.MOE_EUNSUPPORTED and mm(4, 12, 32, M.T_BF16) == M.MOE_EUNSUPPORTED
    assert mm(4, 8, 131072, M.T_BF16) == M.MOE_EUNSUPPORTED and mm(4, 8, 32, 7) == M.MOE_EUNSUPPORTED
    assert mm(4, 8, 32, M.T_BF16, xs=None) == M.MOE_EINVAL and mm(4, 8, 32, M.T_BF16, x=P + 1) == M.MOE_EINVAL
    assert b"moe_int8_mm" in L.moe_last_error() and mm(0, 8, 32, M.T_BF16) == M.MOE_OK
    g = lambda first, E: L.moe_grouped_int8_mm(P, P, 4, None, P, P, first, E, 4, 8, 32, M.T_BF16, P, None, 0, None)  # noqa: E731
    assert g(None, 2) == M.MOE_EINVAL and g(P, 1025) == M.MOE_EUNSUPPORTED


def test_group_refusals():
    L = _lib.load()
    g = lambda T, k, E, ids=P, sc=P, sb=1 << 20, first=P: L.moe_group_routes(ids, T, k, E, first, P, P, P, sc, sb, None)  # noqa: E731
    assert g(-1, 2, 4) == M.MOE_EINVAL and g(4, 0, 4) == M.MOE_EINVAL and g(4, 65, 4) == M.MOE_EINVAL
    assert g(4, 2, 0) == M.MOE_EINVAL and g(4, 2, 1025) == M.MOE_EUNSUPPORTED
    assert g(1 << 29, 4, 8) == M.MOE_EUNSUPPORTED
    assert g(4, 2, 4, ids=None) == M.MOE_EINVAL and g(0, 2, 4, first=None) == M.MOE_EINVAL
    assert g(4096, 2, 4, sc=None) == M.MOE_EINVAL and g(4096, 2, 4, sb=64) == M.MOE_ESCRATCH
    assert L.moe_group_routes_scratch_bytes(4, 2, 8) == 0
    assert L.moe_group_routes_scratch_bytes(-4, 2, 8) == 0


def test_scratch_size_of_refused_products_is_zero():
    for args in [(0, 4, 64, 64, 64), (M.MM_DW, 0, 64, 64, 64), (M.MM_DX, 4, -1, 64, 64), (M.MM_INT8, 1, 4, 0, 64),
                 (9, 4, 64, 64, 64)]:
        assert M.mm_scratch_bytes(*args) == 0


def test_binding_checks():
    bf, f32, i32, i8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
    x, w, first = torch.zeros(6, 16, dtype=bf), torch.zeros(2, 8, 16, dtype=bf), torch.zeros(3, dtype=i32)
    dy = torch.zeros(6, 8, dtype=bf)
    for call, exc, text in [
        (lambda: M.grouped_mm(None, w, first), ValueError, "x must be"),
        (lambda: M.grouped_mm(x.float(), w, first), TypeError, "x: expected"),
        (lambda: M.grouped_mm(x, w.half(), first), TypeError, "w: expected"),
        (lambda: M.grouped_mm(x, w[:, :, :8], first), ValueError, "w: expected shape"),
        (lambda: M.grouped_mm(x, w, first[:2]), ValueError, "first: expected shape"),
        (lambda: M.grouped_mm(x, w, first.long()), TypeError, "first"),
        (lambda: M.grouped_mm(x, w, first, rows=torch.zeros(4)), TypeError, "rows"),
        (lambda: M.grouped_mm(x, w, first, out_dtype=torch.float16), TypeError, "out_dtype"),
        (lambda: M.grouped_mm(x, w, first, out=torch.zeros(6, 9, dtype=bf)), ValueError, "out: expected shape"),
        (lambda: M.grouped_mm(x, w, first, out=torch.zeros(6, 8), out_dtype=bf), TypeError, "out"),
        (lambda: M.grouped_mm(torch.zeros(16, 6, dtype=bf).t(), w, first), ValueError, "contiguous"),
        (lambda: M.grouped_mm(x, w, first), ValueError, "device tensor"),
        (lambda: M.grouped_mm_dx(x, w, first), ValueError, "w: expected shape"),
        (lambda: M.grouped_mm_dx(dy, w, first), ValueError, "device tensor"),
        (lambda: M.grouped_mm_dw(dy, x[:5], first), ValueError, "x: expected 6 rows"),
        (lambda: M.grouped_mm_dw(dy, x, first, accumulate=True), ValueError, "accumulate"),
        (lambda: M.grouped_mm_dw(dy, x, first, out=torch.zeros(2, 8, 8)), ValueError, "out: expected shape"),
        (lambda: M.grouped_mm_dw(dy, x, first), ValueError, "device tensor"),
        (lambda: M.quant_int8(x.float()), TypeError, "x"),
        (lambda: M.quant_int8(x[0]), ValueError, "2 dimensions"),
        (lambda: M.quant_int8(x), ValueError, "device tensor"),
        (lambda: M.int8_mm(x, torch.zeros(6), w[0], torch.zeros(8)), TypeError, "x: expected"),
        (lambda: M.int8_mm(x.to(i8), torch.zeros(5), w[0].to(i8), torch.zeros(8)), ValueError, "x_scales"),
        (lambda: M.int8_mm(x.to(i8), torch.zeros(6), w[0].to(i8), torch.zeros(8), out_dtype=i32), TypeError, "out_dtype"),
        (lambda: M.grouped_int8_mm(x.to(i8), torch.zeros(6), w.to(i8), torch.zeros(8), first), ValueError, "w_scales"),
        (lambda: M.grouped_int8_mm(x.to(i8), torch.zeros(6), w.to(i8), torch.zeros(2, 8), first), ValueError, "device"),
        (lambda: M.group_routes(torch.zeros(4, 2), 8), TypeError, "topk_ids"),
        (lambda: M.group_routes(torch.zeros(4, dtype=i32), 8), ValueError, "2 dimensions"),
        (lambda: M.group_routes(torch.zeros(4, 2, dtype=i32), 8), ValueError, "device tensor"),
    ]:
        with pytest.raises(exc) as ei:
            call()
        assert text in str(ei.value), str(ei.value)


def test_overlapping_buffers_are_refused():
    """64 rows of 64 bf16 values are 8192 bytes; four experts of 64 x 64, 32768."""
    L = _lib.load()
    far = lambda i: P + (i << 20)  # noqa: E731
    big = (1 << 30) + 1
    assert _mm(L, x=far(0), w=far(1), first=far(2), out=far(0) + 8176) == M.MOE_EINVAL
    assert b"overlaps an input" in L.moe_last_error()
    assert _mm(L, x=far(0), w=far(1), first=far(2), out=far(1) + 32752) == M.MOE_EINVAL
    assert _mm(L, x=far(0), w=far(1), first=far(2), out=far(2) - 8176) == M.MOE_EINVAL
    assert _mm(L, x=far(0), w=far(1), first=far(2), rows=far(3) + 252, out=far(3)) == M.MOE_EINVAL
    assert _mm(L, x=far(0), w=far(1), first=far(2), out=far(3), R=big, x_rows=big) == M.MOE_EUNSUPPORTED
    assert L.moe_grouped_mm_dx(M.T_BF16, far(0), far(1), far(2), 4, 64, 64, 64, M.T_BF16, far(0), None, 0, None) == M.MOE_EINVAL
    assert L.moe_grouped_mm_dw(M.T_BF16, far(0), far(1), 64, None, far(2), 4, 64, 64, 64, M.T_FP32, 0, far(1) - 65536 + 16,
                               None, 0, None) == M.MOE_EINVAL
    assert L.moe_quant_int8(M.T_BF16, far(0), 64, 64, far(0), far(1), None) == M.MOE_EINVAL
    assert L.moe_quant_int8(M.T_BF16, far(0), 64, 64, far(1), far(1) + 4092, None) == M.MOE_EINVAL
    assert b"outputs" in L.moe_last_error()
    assert L.moe_int8_mm(far(0), far(1), far(2), far(3), 64, 64, 64, M.T_BF16, far(3) + 240, None, 0, None) == M.MOE_EINVAL
    assert L.moe_group_routes(far(0), 8, 2, 4, far(1), far(0) + 60, far(2), far(3), None, 0, None) == M.MOE_EINVAL
    assert L.moe_group_routes(far(0), 8, 2, 4, far(1), far(2), far(2), far(3), None, 0, None) == M.MOE_EINVAL


def test_scratch_over_buffers_is_refused():
    """Only what a call writes counts: 64 rows need none, 300 rows of a split reduction do."""
    L = _lib.load()
    far = lambda i: (1 << 30) + (i << 28)  # noqa: E731
    need = M.mm_scratch_bytes(M.MM_FORWARD, 1, 300, 64, 8192)
    assert need > 0 and M.mm_scratch_bytes(M.MM_FORWARD, 1, 64, 64, 64) == 0
    call = lambda scratch, nbytes: L.moe_grouped_mm(M.T_BF16, far(0), 300, None, far(1), far(2), 1, 300, 64, 8192,  # noqa: E731
                                                    M.T_BF16, far(3), scratch, nbytes, None)
    assert call(None, 0) == M.MOE_EINVAL and call(far(4), need - 1) == M.MOE_ESCRATCH
    assert call(far(3) - need + 16, need) == M.MOE_EINVAL and b"overlap" in L.moe_last_error()
    assert call(far(1), need) == M.MOE_EINVAL and b"overlaps an input" in L.moe_last_error()


def test_operands_that_require_grad_are_refused_while_autograd_records():
    """The calls return results without a history: with autograd on, gradients would go missing silently."""
    bf, i8 = torch.bfloat16, torch.int8
    g = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype, requires_grad=True)  # noqa: E731
    x, w, dy, first = torch.zeros(6, 16, dtype=bf), torch.zeros(2, 8, 16, dtype=bf), torch.zeros(6, 8, dtype=bf), torch.zeros(3, dtype=torch.int32)
    xq, wq, xs, ws = x.to(i8), w.to(i8), torch.zeros(6), torch.zeros(2, 8)
    calls = [("x", lambda: M.grouped_mm(g(6, 16), w, first)), ("w", lambda: M.grouped_mm(x, g(2, 8, 16), first)),
             ("out", lambda: M.grouped_mm(x, w, first, out=g(6, 8))),
             ("dy", lambda: M.grouped_mm_dx(g(6, 8), w, first)), ("w", lambda: M.grouped_mm_dx(dy, g(2, 8, 16), first)),
             ("dy", lambda: M.grouped_mm_dw(g(6, 8), x, first)), ("x", lambda: M.grouped_mm_dw(dy, g(6, 16), first)),
             ("out", lambda: M.grouped_mm_dw(dy, x, first, out=g(2, 8, 16, dtype=torch.float32), accumulate=True)),
             ("x", lambda: M.quant_int8(g(6, 16))), ("scales", lambda: M.quant_int8(x, scales=g(6, dtype=torch.float32))),
             ("x_scales", lambda: M.int8_mm(xq, g(6, dtype=torch.float32), wq[0], ws[0])),
             ("w_scales", lambda: M.grouped_int8_mm(xq, xs, wq, g(2, 8, dtype=torch.float32), first))]
    for name, call in calls:
        with pytest.raises(ValueError, match=f"^{name} requires grad"):
            call()
        for off in (torch.no_grad(), torch.inference_mode()):
            with off, pytest.raises(ValueError, match="device tensor"):
                call()


def test_plan_query():
    """The shape a product runs with; refused sizes as the products refuse them."""
    L = _lib.load()
    assert M.debug_mm_plan(M.MM_FORWARD, 384, 48, 1152, 7168) == (16, 16, 1)
    rows, cols, splits = M.debug_mm_plan(M.MM_DW, 3, 8001, 72, 136)
    assert (rows, cols) == (128, 128) and splits > 1
    assert M.mm_scratch_bytes(M.MM_DW, 3, 8001, 72, 136) == splits * 3 * 72 * 136 * 4
    for args, code in [((0, 4, 64, 64, 64), M.MOE_EINVAL), ((9, 4, 64, 64, 64), M.MOE_EINVAL), ((1, 4, 0, 64, 64), M.MOE_EINVAL),
                       ((1, 4, 64, 60, 64), M.MOE_EUNSUPPORTED), ((4, 4, 64, 64, 24), M.MOE_EUNSUPPORTED)]:
        with pytest.raises(M.MoeError, match="moe_debug_mm_plan") as e:
            M.debug_mm_plan(*args)
        assert e.value.code == code
    one = C.c_int()
    assert L.moe_debug_mm_plan(M.MM_DX, 4, 64, 64, 64, C.byref(one), None, C.byref(one)) == M.MOE_EINVAL
