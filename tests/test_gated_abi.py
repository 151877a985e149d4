"""Refusals of the gated block, the 8-bit floating-point products and their quantiser, on the host: nothing here
launches GPU work."""
import ctypes as C

import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from block_scaled_fp4_histogram_amd import _lib

P = 4096   # an aligned address that is never read


def far(i):
    return (1 << 30) + (i << 24)


def _form(**kw):
    a = dict(activation=M.ACT_SWIGLU, layout=M.W13_UP_GATE, limit=0.0, alpha=1.0, beta=0.0)
    a.update(kw)
    return C.addressof(_keep.setdefault(str(sorted(a.items(), key=str)), _lib.GluForm(*a.values())))


_keep = {}


def _glu(L, **kw):
    a = dict(dtype=M.T_BF16, x=far(0), x_rows=64, rows=None, w=far(1), first=far(2), E=4, R=64, I=64, K=64, form=None,
             out_dtype=M.T_BF16, h=far(3), pre=None, scratch=None, bytes=0)
    a.update(kw)
    return L.moe_grouped_glu(*a.values(), None)


FORM_CASES = [(dict(activation=M.ACT_RELU2_NO_MUL), M.MOE_EUNSUPPORTED), (dict(activation=9), M.MOE_EUNSUPPORTED),
              (dict(layout=2), M.MOE_EINVAL), (dict(alpha=float("inf")), M.MOE_EINVAL), (dict(beta=float("nan")), M.MOE_EINVAL),
              (dict(activation=M.ACT_SITU, limit=7.0), M.MOE_EUNSUPPORTED), (dict(activation=M.ACT_SITU, alpha=1.5), M.MOE_EUNSUPPORTED),
              (dict(activation=M.ACT_SITU, beta=1.0), M.MOE_EUNSUPPORTED)]


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=M.T_FP32), M.MOE_EUNSUPPORTED), (dict(out_dtype=M.T_FP16), M.MOE_EUNSUPPORTED), (dict(I=60), M.MOE_EUNSUPPORTED),
    (dict(K=65), M.MOE_EUNSUPPORTED), (dict(I=0), M.MOE_EINVAL), (dict(K=-8), M.MOE_EINVAL), (dict(R=-1), M.MOE_EINVAL),
    (dict(E=0), M.MOE_EINVAL), (dict(E=1025), M.MOE_EUNSUPPORTED), (dict(I=(1 << 19) + 8), M.MOE_EUNSUPPORTED),
    (dict(K=(1 << 20) + 8), M.MOE_EUNSUPPORTED), (dict(x=None), M.MOE_EINVAL), (dict(w=P + 8), M.MOE_EINVAL),
    (dict(h=P + 2), M.MOE_EINVAL), (dict(pre=P + 2), M.MOE_EINVAL), (dict(first=None), M.MOE_EINVAL), (dict(first=P + 2), M.MOE_EINVAL),
    (dict(rows=P + 1), M.MOE_EINVAL), (dict(x_rows=63), M.MOE_EINVAL), (dict(x_rows=-1, rows=P), M.MOE_EINVAL),
    (dict(R=(1 << 30) + 1, x_rows=1 << 31), M.MOE_EUNSUPPORTED),
    (dict(h=far(0) + 8176), M.MOE_EINVAL), (dict(h=far(1) + 65520), M.MOE_EINVAL), (dict(pre=far(3) + 8176), M.MOE_EINVAL),
    (dict(pre=far(2) - 16368), M.MOE_EINVAL), (dict(rows=far(3) + 252), M.MOE_EINVAL),
    (dict(R=300, x_rows=300, I=64, K=8192, E=1, w=far(9)), M.MOE_EINVAL),   # a split reduction without scratch
    (dict(R=0), M.MOE_OK), (dict(R=0, x=None, h=None), M.MOE_OK), (dict(R=0, E=1, first=None), M.MOE_OK)])
def test_forward_refusals(kw, code):
    L = _lib.load()
    assert _glu(L, **kw) == code
    if code != M.MOE_OK:
        assert L.moe_last_error().decode().startswith("moe_grouped_glu" if kw.get("first", P) else "moe_glu")


@pytest.mark.parametrize("form,code", FORM_CASES)
def test_form_refusals(form, code):
    L = _lib.load()
    f = _form(**form)
    assert _glu(L, form=f) == code
    assert L.moe_grouped_glu_dx(M.T_BF16, P, P, P, P, 4, 64, 64, 64, f, P, None, None, 0, None) == code
    assert L.moe_glu_grad(M.T_BF16, P, P, 4, 64, f, P, None, None) == code
    assert L.moe_grouped_fp8_glu(P, P, 64, None, P, P, P, 4, 64, 64, 64, f, M.T_BF16, P, None, 0, None) == code


def test_backward_refusals():
    L = _lib.load()

    def dx(dtype=M.T_BF16, dy=far(0), w=far(1), pre=far(2), first=far(3), E=4, R=64, N=64, I=64, d_pre=far(4), h=None):
        return L.moe_grouped_glu_dx(dtype, dy, w, pre, first, E, R, N, I, None, d_pre, h, None, 0, None)

    for kw, code in [(dict(dtype=M.T_FP32), M.MOE_EUNSUPPORTED), (dict(N=12), M.MOE_EUNSUPPORTED), (dict(I=12), M.MOE_EUNSUPPORTED),
                     (dict(I=(1 << 19) + 8), M.MOE_EUNSUPPORTED), (dict(E=1025), M.MOE_EUNSUPPORTED), (dict(R=-1), M.MOE_EINVAL),
                     (dict(dy=None), M.MOE_EINVAL), (dict(w=None), M.MOE_EINVAL), (dict(pre=None), M.MOE_EINVAL),
                     (dict(d_pre=None), M.MOE_EINVAL), (dict(d_pre=P + 8), M.MOE_EINVAL), (dict(h=P + 8), M.MOE_EINVAL),
                     (dict(first=None), M.MOE_EINVAL), (dict(first=P + 2), M.MOE_EINVAL), (dict(d_pre=far(2)), M.MOE_EINVAL),
                     (dict(d_pre=far(0) - 16368), M.MOE_EINVAL), (dict(h=far(4) + 16368), M.MOE_EINVAL),
                     (dict(R=300, E=1, N=8192), M.MOE_EINVAL), (dict(R=0), M.MOE_OK), (dict(R=0, dy=None, d_pre=None), M.MOE_OK)]:
        assert dx(**kw) == code, kw

    def grad(dtype=M.T_BF16, dh=far(0), pre=far(1), R=4, I=64, d_pre=far(2), h=None):
        return L.moe_glu_grad(dtype, dh, pre, R, I, None, d_pre, h, None)

    for kw, code in [(dict(dtype=M.T_FP32), M.MOE_EUNSUPPORTED), (dict(I=12), M.MOE_EUNSUPPORTED), (dict(I=0), M.MOE_EINVAL),
                     (dict(R=-1), M.MOE_EINVAL), (dict(R=(1 << 30) + 1), M.MOE_EUNSUPPORTED), (dict(dh=None), M.MOE_EINVAL),
                     (dict(pre=P + 4), M.MOE_EINVAL), (dict(d_pre=None), M.MOE_EINVAL), (dict(h=P + 2), M.MOE_EINVAL),
                     (dict(d_pre=far(1)), M.MOE_EINVAL), (dict(h=far(0)), M.MOE_EINVAL), (dict(h=far(2)), M.MOE_EINVAL),
                     (dict(R=0, dh=None), M.MOE_OK)]:
        assert grad(**kw) == code, kw
        if code != M.MOE_OK:
            assert L.moe_last_error().startswith(b"moe_glu_grad")


def test_fp8_refusals():
    L = _lib.load()

    def quant(dtype=M.T_BF16, x=far(0), rows=4, cols=64, q=far(1), s=far(2)):
        return L.moe_quant_fp8(dtype, x, rows, cols, q, s, None)

    for kw, code in [(dict(dtype=M.T_FP32), M.MOE_EUNSUPPORTED), (dict(cols=24), M.MOE_EUNSUPPORTED), (dict(cols=0), M.MOE_EINVAL),
                     (dict(cols=(1 << 20) + 16), M.MOE_EUNSUPPORTED), (dict(rows=-1), M.MOE_EINVAL), (dict(x=P + 4), M.MOE_EINVAL),
                     (dict(q=None), M.MOE_EINVAL), (dict(s=None), M.MOE_EINVAL), (dict(s=P + 2), M.MOE_EINVAL),
                     (dict(q=far(0)), M.MOE_EINVAL), (dict(s=far(1) + 252), M.MOE_EINVAL), (dict(rows=0, x=None), M.MOE_OK)]:
        assert quant(**kw) == code, kw

    def mm(glu, x=far(0), xs=far(1), x_rows=64, rows=None, w=far(2), ws=far(3), first=far(4), E=4, R=64, N=64, K=64, od=M.T_BF16,
           out=far(5)):
        a = (x, xs, x_rows, rows, w, ws, first, E, R, N, K)
        return (L.moe_grouped_fp8_glu(*a, None, od, out, None, 0, None) if glu else
                L.moe_grouped_fp8_mm(*a, od, out, None, 0, None))

    for glu in (False, True):
        for kw, code in [(dict(K=24), M.MOE_EUNSUPPORTED), (dict(N=12), M.MOE_EUNSUPPORTED), (dict(od=7), M.MOE_EUNSUPPORTED),
                         (dict(E=1025), M.MOE_EUNSUPPORTED), (dict(R=-1), M.MOE_EINVAL), (dict(xs=None), M.MOE_EINVAL),
                         (dict(ws=None), M.MOE_EINVAL), (dict(ws=P + 2), M.MOE_EINVAL), (dict(x=P + 1), M.MOE_EINVAL),
                         (dict(first=None), M.MOE_EINVAL), (dict(x_rows=63), M.MOE_EINVAL), (dict(rows=P + 2), M.MOE_EINVAL),
                         (dict(out=far(0) + 4080), M.MOE_EINVAL), (dict(out=far(1) + 240), M.MOE_EINVAL),
                         (dict(out=far(3)), M.MOE_EINVAL), (dict(out=far(4)), M.MOE_EINVAL), (dict(R=0), M.MOE_OK),
                         (dict(R=300, x_rows=300, E=1, K=8192), M.MOE_EINVAL), (dict(R=0, first=None, E=1), M.MOE_OK)]:
            assert mm(glu, **kw) == code, (glu, kw)
    assert mm(False, N=(1 << 20)) == M.MOE_EINVAL and mm(True, N=(1 << 20)) == M.MOE_EUNSUPPORTED   # overlap; two branches


def test_scratch_and_plans():
    for op in (M.MM_GLU, M.MM_GLU_DX, M.MM_FP8, M.MM_FP8_GLU):
        assert M.mm_scratch_bytes(op, 4, 64, 0, 64) == 0 and M.mm_scratch_bytes(op, 0, 64, 64, 64) == 0
        assert M.mm_scratch_bytes(op, 4, 0, 64, 64) == 0
        rows, cols, splits = M.debug_mm_plan(op, 1, 300, 64 if op != M.MM_GLU_DX else 8192, 8192 if op != M.MM_GLU_DX else 64)
        n = 128 if op in (M.MM_GLU, M.MM_FP8_GLU) else 64
        assert splits > 1
        assert M.mm_scratch_bytes(op, 1, 300, 64 if op != M.MM_GLU_DX else 8192, 8192 if op != M.MM_GLU_DX else 64) == splits * 300 * n * 4
    assert M.debug_mm_plan(M.MM_GLU, 384, 48, 576, 7168) == (16, 8, 1)
    assert M.debug_mm_plan(M.MM_FP8, 384, 48, 1152, 7168) == (16, 16, 1)
    for args in [(M.MM_FP8, 4, 64, 64, 24), (M.MM_FP8_GLU, 4, 64, 64, 24), (M.MM_GLU, 4, 64, 1 << 20, 64), (M.MM_GLU_DX, 4, 64, 64, 1 << 20)]:
        with pytest.raises(M.MoeError) as e:
            M.debug_mm_plan(*args)
        assert e.value.code == M.MOE_EUNSUPPORTED


def _tensors():
    bf, i32, f8 = torch.bfloat16, torch.int32, torch.float8_e4m3fn
    t = dict(x=torch.zeros(6, 16, dtype=bf), w=torch.zeros(2, 16, 16, dtype=bf), first=torch.zeros(3, dtype=i32),
             dy=torch.zeros(6, 16, dtype=bf), wd=torch.zeros(2, 16, 8, dtype=bf), pre=torch.zeros(6, 16, dtype=bf),
             dh=torch.zeros(6, 8, dtype=bf))
    t.update(xq=t["x"].to(f8), xs=torch.zeros(6, 1), wq=t["w"].to(f8), ws=torch.zeros(2, 1, 1), wgs=torch.zeros(2, 2, 1, 1))
    return t


def test_binding_checks():
    t = _tensors()
    x, w, first, dy, wd, pre, dh, xq, xs, wq, ws, wgs = t.values()
    for call, exc, text in [
        (lambda: M.glu(None, w[0]), ValueError, "x must be"), (lambda: M.glu(x.float(), w[0]), TypeError, "x: expected"),
        (lambda: M.glu(x, w), ValueError, "w must be"), (lambda: M.glu(x, w[0].half()), TypeError, "w: expected"),
        (lambda: M.glu(x, w[0, :15]), ValueError, "two branches"), (lambda: M.glu(x, w[0, :, :8]), ValueError, "w: expected shape"),
        (lambda: M.glu(x, w[0], out=torch.zeros(6, 9, dtype=torch.bfloat16)), ValueError, "out: expected shape"),
        (lambda: M.glu(x, w[0], pre=torch.zeros(6, 8, dtype=torch.bfloat16)), ValueError, "pre: expected shape"),
        (lambda: M.glu(x, w[0], pre=torch.zeros(6, 16)), TypeError, "pre: expected"),
        (lambda: M.glu(x, w[0], out_dtype=torch.float16), TypeError, "out_dtype"),
        (lambda: M.glu(x, w[0], limit="7"), TypeError, "number"), (lambda: M.glu(x, w[0], activation=1.5), TypeError, "int"),
        (lambda: M.glu(x, w[0]), ValueError, "device tensor"),
        (lambda: M.glu(torch.zeros(16, 6, dtype=torch.bfloat16).t(), w[0]), ValueError, "contiguous"),
        (lambda: M.grouped_glu(x, w, None), ValueError, "first is required"),
        (lambda: M.grouped_glu(x, w[0], first), ValueError, "w must be"), (lambda: M.grouped_glu(x, w, first[:2]), ValueError, "first: expected shape"),
        (lambda: M.grouped_glu(x, w, first, rows=torch.zeros(4)), TypeError, "rows"),
        (lambda: M.grouped_glu(x, w, first), ValueError, "device tensor"),
        (lambda: M.glu_dx(dy, wd[0], pre[:5]), ValueError, "pre: expected shape"), (lambda: M.glu_dx(dy, wd, pre), ValueError, "w must be"),
        (lambda: M.glu_dx(dy, wd[0], pre.float()), TypeError, "pre: expected"), (lambda: M.glu_dx(dy, wd[0], pre), ValueError, "device tensor"),
        (lambda: M.glu_dx(dy, wd[0], pre, h=torch.zeros(6, 16, dtype=torch.bfloat16)), ValueError, "h: expected shape"),
        (lambda: M.grouped_glu_dx(dy, wd, pre, None), ValueError, "first is required"),
        (lambda: M.grouped_glu_dx(dy, wd, pre, first), ValueError, "device tensor"),
        (lambda: M.glu_grad(dh, pre[:, :8]), ValueError, "pre: expected shape"), (lambda: M.glu_grad(dh.float(), pre), TypeError, "dh: expected"),
        (lambda: M.glu_grad(dh, pre, out=torch.zeros(6, 16)), TypeError, "out: expected"), (lambda: M.glu_grad(dh, pre), ValueError, "device tensor"),
        (lambda: M.quant_fp8(x.float()), TypeError, "x: expected"), (lambda: M.quant_fp8(x, out=x), TypeError, "out: expected torch.float8_e4m3fn"),
        (lambda: M.quant_fp8(x, scales=torch.zeros(6)), ValueError, "scales: expected shape"), (lambda: M.quant_fp8(x), ValueError, "device tensor"),
        (lambda: M.fp8_mm(x, xs, wq[0], ws[0]), TypeError, "x: expected"), (lambda: M.fp8_mm(xq, xs[:5], wq[0], ws[0]), ValueError, "x_scales"),
        (lambda: M.fp8_mm(xq, xs, wq[0], ws), ValueError, "w_scales: expected shape"),
        (lambda: M.fp8_mm(xq, xs, wq[0].view(torch.float8_e5m2), ws[0]), TypeError, "w: expected"),
        (lambda: M.fp8_mm(xq, xs, wq[0], ws[0], out_dtype=torch.int32), TypeError, "out_dtype"),
        (lambda: M.fp8_mm(xq, xs, wq[0], ws[0]), ValueError, "device tensor"),
        (lambda: M.grouped_fp8_mm(xq, xs, wq, ws, None), ValueError, "first is required"),
        (lambda: M.grouped_fp8_mm(xq, xs, wq, ws[0], first), ValueError, "w_scales"), (lambda: M.grouped_fp8_mm(xq, xs, wq, ws, first), ValueError, "device"),
        (lambda: M.fp8_glu(xq, xs, wq[0], ws[0]), ValueError, "w_scales: expected shape"), (lambda: M.fp8_glu(xq, xs, wq[0, :15], wgs[0]), ValueError, "two branches"),
        (lambda: M.fp8_glu(xq, xs, wq[0], wgs[0]), ValueError, "device tensor"),
        (lambda: M.grouped_fp8_glu(xq, xs, wq, wgs, first, rows=first.long()), TypeError, "rows"),
        (lambda: M.grouped_fp8_glu(xq, xs, wq, wgs, first), ValueError, "device tensor"),
    ]:
        with pytest.raises(exc) as ei:
            call()
        assert text in str(ei.value), str(ei.value)


def test_operands_that_require_grad_are_refused_while_autograd_records():
    t = _tensors()
    x, w, first, dy, wd, pre, dh, xq, xs, wq, ws, wgs = t.values()
    g = lambda v: v.clone().requires_grad_()  # noqa: E731
    for name, call in [("x", lambda: M.glu(g(x), w[0])), ("w", lambda: M.grouped_glu(x, g(w), first)), ("pre", lambda: M.glu(x, w[0], pre=g(pre))),
                       ("dy", lambda: M.glu_dx(g(dy), wd[0], pre)), ("w", lambda: M.grouped_glu_dx(dy, g(wd), pre, first)),
                       ("pre", lambda: M.glu_grad(dh, g(pre))), ("h", lambda: M.glu_grad(dh, pre, h=g(dh))), ("x", lambda: M.quant_fp8(g(x))),
                       ("x_scales", lambda: M.fp8_mm(xq, g(xs), wq[0], ws[0])), ("w_scales", lambda: M.grouped_fp8_glu(xq, xs, wq, g(wgs), first))]:
        with pytest.raises(ValueError, match=f"^{name} requires grad"):
            call()
        for off in (torch.no_grad(), torch.inference_mode()):
            with off, pytest.raises(ValueError, match="device tensor"):
                call()
