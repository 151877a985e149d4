"""MOE_FP8_FAST_SUMS at the C ABI and the binding, on the host: nothing here launches GPU work."""
import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from block_scaled_fp4_histogram_amd import _lib

P = 4096   # an aligned address that is never read
FAST = M.FP8_FAST_SUMS


def test_result_types():
    L = _lib.load()
    for od, code in [(M.T_BF16, M.MOE_OK), (M.T_BF16 | FAST, M.MOE_OK), (M.T_FP16 | FAST, M.MOE_OK), (M.T_FP32, M.MOE_OK),
                     (M.T_FP32 | FAST, M.MOE_EUNSUPPORTED), (FAST, M.MOE_EUNSUPPORTED), (2 * FAST | M.T_BF16, M.MOE_EUNSUPPORTED),
                     (-1, M.MOE_EUNSUPPORTED), (M.T_BF16 | FAST | -1 << 31, M.MOE_EUNSUPPORTED)]:
        args = (P, P, 64, None, P, P, P, 4, 0, 64, 64)   # no rows
        assert L.moe_grouped_fp8_mm(*args, od, P, None, 0, None) == code, od
        assert L.moe_grouped_fp8_glu(*args, None, od, P, None, 0, None) == code, od
    # no other call knows it
    assert L.moe_grouped_mm(M.T_BF16, P, 64, None, P, P, 4, 0, 64, 64, M.T_BF16 | FAST, P, None, 0, None) == M.MOE_EUNSUPPORTED
    assert L.moe_grouped_int8_mm(P, P, 64, None, P, P, P, 4, 0, 64, 64, M.T_BF16 | FAST, P, None, 0, None) == M.MOE_EUNSUPPORTED


def test_scratch_and_plans():
    for op in (M.MM_FP8, M.MM_FP8_GLU):
        n = 128 if op == M.MM_FP8_GLU else 64
        splits = M.debug_mm_plan(op | FAST, 1, 300, 64, 8192)[2]
        assert splits > 1 and M.mm_scratch_bytes(op | FAST, 1, 300, 64, 8192) == splits * 300 * n * 4
        assert M.debug_mm_plan(op | FAST, 384, 48, 576, 7168) == M.debug_mm_plan(op, 384, 48, 576, 7168)   # streamed
        # a call with fast sums needs the scratch of its own plan
        L = _lib.load()
        args = (P, P, 300, None, P, P, None, 1, 300, 64, 8192)
        call = (lambda s, b: L.moe_grouped_fp8_glu(*args, None, M.T_BF16 | FAST, 1 << 30, s, b, None)) if op == M.MM_FP8_GLU else (
            lambda s, b: L.moe_grouped_fp8_mm(*args, M.T_BF16 | FAST, 1 << 30, s, b, None))
        assert call(None, 0) == M.MOE_EINVAL and call(P, splits * 300 * n * 4 - 1) == M.MOE_ESCRATCH
    for op in (M.MM_FORWARD, M.MM_INT8, M.MM_GLU):
        assert M.mm_scratch_bytes(op | FAST, 1, 300, 64, 8192) == 0
        with pytest.raises(M.MoeError) as e:
            M.debug_mm_plan(op | FAST, 1, 300, 64, 8192)
        assert e.value.code == M.MOE_EINVAL


def test_fp32_results_are_refused_by_the_binding():
    f8 = torch.float8_e4m3fn
    xq, xs, wq, ws = torch.zeros(6, 16).to(f8), torch.zeros(6, 1), torch.zeros(16, 16).to(f8), torch.zeros(1, 1)
    with pytest.raises(TypeError, match="fast_sums"):
        M.fp8_mm(xq, xs, wq, ws, out_dtype=torch.float32, fast_sums=True)
    with pytest.raises(TypeError, match="fast_sums"):
        M.fp8_glu(xq, xs, wq, torch.zeros(2, 1, 1), out_dtype=torch.float32, fast_sums=True)
    with pytest.raises(ValueError, match="device tensor"):
        M.fp8_mm(xq, xs, wq, ws, fast_sums=True)
