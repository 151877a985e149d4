// C ABI of the ragged expert products, the 8-bit integer products and the
// route grouping (declared in include/moe.h): argument validation and launches.
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>

#include "moe.h"
#include "moe_common.h"
#include "moe_mm.h"

namespace {

int fail(int code, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return moe::set_error(code, buf);
}

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int launched(hipError_t e, const char *what) {
  return e == hipSuccess ? MOE_OK : fail(MOE_EHIP, "%s: %s", what, hipGetErrorString(e));
}

// Longest row (elements) of the products: a tile's rows stay within 32-bit byte offsets.
constexpr int kMmMaxDim = 1 << 20;
// Most rows: row numbers a tile past the last one stay within 32 bits.
constexpr int kMmMaxRows = 1 << 30;
// Longest int8 reduction: (-128)^2 a term in a 32-bit sum.
constexpr int kI8MaxK = 131056;

int check_shape(const char *fn, int unit, const int32_t *first, int E, int R, int N, int K) {
  if (R < 0) return fail(MOE_EINVAL, "%s: rows R=%d", fn, R);
  if (N < 1 || K < 1) return fail(MOE_EINVAL, "%s: N=%d, K=%d", fn, N, K);
  if (E < 1) return fail(MOE_EINVAL, "%s: E=%d", fn, E);
  if (!aligned(first, 4)) return fail(MOE_EINVAL, "%s: first needs 4-byte alignment", fn);
  if (E > moe::kMaxExperts) return fail(MOE_EUNSUPPORTED, "%s: E=%d above %d", fn, E, moe::kMaxExperts);
  if (N % 8 || K % unit) return fail(MOE_EUNSUPPORTED, "%s: N=%d must be a multiple of 8, K=%d of %d", fn, N, K, unit);
  if (N > kMmMaxDim || K > kMmMaxDim) return fail(MOE_EUNSUPPORTED, "%s: N=%d or K=%d above %d", fn, N, K, kMmMaxDim);
  if (R > kMmMaxRows) return fail(MOE_EUNSUPPORTED, "%s: R=%d above %d", fn, R, kMmMaxRows);
  return MOE_OK;
}

int check_16bit(const char *fn, int dtype, int out_dtype) {
  if (dtype != MOE_T_BF16 && dtype != MOE_T_FP16) return fail(MOE_EUNSUPPORTED, "%s: dtype %d is not bf16 or fp16", fn, dtype);
  if (out_dtype != dtype && out_dtype != MOE_T_FP32)
    return fail(MOE_EUNSUPPORTED, "%s: out_dtype %d is neither the operands' type nor fp32", fn, out_dtype);
  return MOE_OK;
}

int check_ptrs(const char *fn, const void *const *p, int n) {
  for (int i = 0; i < n; i++)
    if (!p[i] || !aligned(p[i], 16)) return fail(MOE_EINVAL, "%s: null or misaligned pointer (16 bytes)", fn);
  return MOE_OK;
}

int check_rows(const char *fn, const int32_t *rows, long long x_rows, int R) {
  if (!aligned(rows, 4)) return fail(MOE_EINVAL, "%s: rows needs 4-byte alignment", fn);
  if (x_rows < 0 || (!rows && x_rows < R)) return fail(MOE_EINVAL, "%s: x_rows=%lld for R=%d rows", fn, x_rows, R);
  return MOE_OK;
}

// Buffers of a call: what it writes overlaps neither what it reads nor each other.
struct Span {
  const void *p;
  size_t bytes;
};

// `work`: the part of the scratch that the call writes.
int check_scratch(const char *fn, int op, int E, int R, int N, int K, const void *scratch, size_t bytes, Span *work) {
  const size_t need = moe_mm_scratch_bytes(op, E, R, N, K);
  if (need && (!scratch || !aligned(scratch, 16))) return fail(MOE_EINVAL, "%s: null or misaligned scratch (16 bytes)", fn);
  if (bytes < need) return fail(MOE_ESCRATCH, "%s: scratch holds %zu bytes, %zu needed", fn, bytes, need);
  *work = {need ? scratch : nullptr, need};
  return MOE_OK;
}

int check_apart(const char *fn, std::initializer_list<Span> written, std::initializer_list<Span> read) {
  auto meet = [](const Span &a, const Span &b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x && y && x < y + b.bytes && y < x + a.bytes;
  };
  for (const Span *w = written.begin(); w != written.end(); w++) {
    for (const Span &r : read)
      if (meet(*w, r)) return fail(MOE_EINVAL, "%s: an output or the scratch overlaps an input", fn);
    for (const Span *v = written.begin(); v != w; v++)
      if (meet(*w, *v)) return fail(MOE_EINVAL, "%s: outputs or the scratch overlap", fn);
  }
  return MOE_OK;
}

int check_op(const char *fn, int op, int E, int R, int N, int K) {
  if (op < MOE_MM_FORWARD || op > MOE_MM_INT8) return fail(MOE_EINVAL, "%s: op=%d", fn, op);
  return check_shape(fn, op == MOE_MM_INT8 ? 16 : 8, nullptr, E, R, N, K);
}

moe::MmPlan plan_of(int op, int E, int R, int N, int K) {
  const bool i8 = op == MOE_MM_INT8;
  return moe::mm_plan(i8 ? MOE_MM_FORWARD : op, i8 ? moe::MM_I8 : moe::MM_BF16, E, R, N, K);
}

size_t type_size(int dtype) { return dtype == MOE_T_FP32 ? 4 : 2; }

}  // namespace

#define TRY(expr)              \
  do {                         \
    const int rc_ = (expr);    \
    if (rc_ != MOE_OK) return rc_; \
  } while (0)

extern "C" {

size_t moe_mm_scratch_bytes(int op, int E, int R, int N, int K) {
  if (check_op("moe_mm_scratch_bytes", op, E, R, N, K) != MOE_OK) return 0;
  return R == 0 ? 0 : plan_of(op, E, R, N, K).scratch;
}

int moe_debug_mm_plan(int op, int E, int R, int N, int K, int *rows, int *cols, int *splits) {
  const char *fn = "moe_debug_mm_plan";
  TRY(check_op(fn, op, E, R, N, K));
  if (R == 0 || !rows || !cols || !splits) return fail(MOE_EINVAL, "%s: R=0 or a null pointer", fn);
  const moe::MmPlan m = plan_of(op, E, R, N, K);
  *rows = m.rows, *cols = m.cols, *splits = m.splits;
  return MOE_OK;
}

int moe_grouped_mm(int dtype, const void *x, long long x_rows, const int32_t *rows, const void *w,
                   const int32_t *first, int E, int R, int N, int K, int out_dtype, void *out, void *scratch,
                   size_t scratch_bytes, void *stream) {
  const char *fn = "moe_grouped_mm";
  TRY(check_16bit(fn, dtype, out_dtype));
  TRY(check_shape(fn, 8, first, E, R, N, K));
  TRY(check_rows(fn, rows, x_rows, R));
  if (R == 0) return MOE_OK;
  if (!first) return fail(MOE_EINVAL, "%s: null first", fn);
  const void *p[] = {w, out, x};   // an x without rows is not read
  TRY(check_ptrs(fn, p, x_rows ? 3 : 2));
  Span work;
  TRY(check_scratch(fn, MOE_MM_FORWARD, E, R, N, K, scratch, scratch_bytes, &work));
  TRY(check_apart(fn, {{out, (size_t)R * N * type_size(out_dtype)}, work},
                  {{x, (size_t)x_rows * K * 2}, {w, (size_t)E * N * K * 2}, {first, (E + 1) * sizeof *first},
                   {rows, R * sizeof *rows}}));
  moe::MmArgs a = {};
  a.part = (float *)scratch;
  a.op = moe::MM_FORWARD, a.type = dtype, a.out_type = out_dtype;
  a.x = x, a.x_rows = (long)x_rows, a.rows = rows, a.w = w, a.first = first;
  a.E = E, a.R = R, a.N = N, a.K = K, a.out = out;
  return launched(moe::launch_mm(a, (hipStream_t)stream), fn);
}

int moe_grouped_mm_dx(int dtype, const void *dy, const void *w, const int32_t *first, int E, int R, int N, int K,
                      int out_dtype, void *dx, void *scratch, size_t scratch_bytes, void *stream) {
  const char *fn = "moe_grouped_mm_dx";
  TRY(check_16bit(fn, dtype, out_dtype));
  TRY(check_shape(fn, 8, first, E, R, N, K));
  if (R == 0) return MOE_OK;
  if (!first) return fail(MOE_EINVAL, "%s: null first", fn);
  const void *p[] = {dy, w, dx};
  TRY(check_ptrs(fn, p, 3));
  Span work;
  TRY(check_scratch(fn, MOE_MM_DX, E, R, N, K, scratch, scratch_bytes, &work));
  TRY(check_apart(fn, {{dx, (size_t)R * K * type_size(out_dtype)}, work},
                  {{dy, (size_t)R * N * 2}, {w, (size_t)E * N * K * 2}, {first, (E + 1) * sizeof *first}}));
  moe::MmArgs a = {};
  a.part = (float *)scratch;
  a.op = moe::MM_DX, a.type = dtype, a.out_type = out_dtype;
  a.dy = dy, a.w = w, a.first = first;
  a.E = E, a.R = R, a.N = N, a.K = K, a.out = dx;
  return launched(moe::launch_mm(a, (hipStream_t)stream), fn);
}

int moe_grouped_mm_dw(int dtype, const void *dy, const void *x, long long x_rows, const int32_t *rows,
                      const int32_t *first, int E, int R, int N, int K, int out_dtype, int accumulate, void *dw,
                      void *scratch, size_t scratch_bytes, void *stream) {
  const char *fn = "moe_grouped_mm_dw";
  TRY(check_16bit(fn, dtype, out_dtype));
  if (accumulate && out_dtype != MOE_T_FP32) return fail(MOE_EUNSUPPORTED, "%s: accumulate needs an fp32 dw", fn);
  TRY(check_shape(fn, 8, first, E, R, N, K));
  TRY(check_rows(fn, rows, x_rows, R));
  if (!first) return fail(MOE_EINVAL, "%s: null first", fn);
  const void *p[] = {dw, dy, x};   // without rows dy and x are not read
  TRY(check_ptrs(fn, p, R == 0 ? 1 : x_rows ? 3 : 2));
  Span work;
  TRY(check_scratch(fn, MOE_MM_DW, E, R, N, K, scratch, scratch_bytes, &work));
  TRY(check_apart(fn, {{dw, (size_t)E * N * K * type_size(out_dtype)}, work},
                  {{dy, (size_t)R * N * 2}, {x, (size_t)x_rows * K * 2}, {first, (E + 1) * sizeof *first},
                   {rows, R * sizeof *rows}}));
  moe::MmArgs a = {};
  a.part = (float *)scratch;
  a.op = moe::MM_DW, a.type = dtype, a.out_type = out_dtype, a.accumulate = accumulate;
  a.dy = dy, a.x = x, a.x_rows = (long)x_rows, a.rows = rows, a.first = first;
  a.E = E, a.R = R, a.N = N, a.K = K, a.out = dw;
  return launched(moe::launch_mm(a, (hipStream_t)stream), fn);
}

int moe_quant_int8(int dtype, const void *x, int rows, int cols, int8_t *q, float *scales, void *stream) {
  const char *fn = "moe_quant_int8";
  if (dtype != MOE_T_BF16 && dtype != MOE_T_FP16) return fail(MOE_EUNSUPPORTED, "%s: dtype %d is not bf16 or fp16", fn, dtype);
  if (rows < 0 || cols < 1) return fail(MOE_EINVAL, "%s: rows=%d, cols=%d", fn, rows, cols);
  if (cols % 16 || cols > kMmMaxDim) return fail(MOE_EUNSUPPORTED, "%s: cols=%d must be a multiple of 16 up to %d", fn, cols, kMmMaxDim);
  if (rows == 0) return MOE_OK;
  const void *p[] = {x, q};
  TRY(check_ptrs(fn, p, 2));
  if (!scales || !aligned(scales, 4)) return fail(MOE_EINVAL, "%s: null or misaligned scales", fn);
  TRY(check_apart(fn, {{q, (size_t)rows * cols}, {scales, rows * sizeof *scales}}, {{x, (size_t)rows * cols * 2}}));
  return launched(moe::launch_quant_int8(dtype, x, rows, cols, q, scales, (hipStream_t)stream), fn);
}

int moe_grouped_int8_mm(const int8_t *x, const float *x_scales, long long x_rows, const int32_t *rows, const int8_t *w,
                        const float *w_scales, const int32_t *first, int E, int R, int N, int K, int out_dtype,
                        void *out, void *scratch, size_t scratch_bytes, void *stream) {
  const char *fn = first ? "moe_grouped_int8_mm" : "moe_int8_mm";
  if (out_dtype != MOE_T_BF16 && out_dtype != MOE_T_FP16 && out_dtype != MOE_T_FP32)
    return fail(MOE_EUNSUPPORTED, "%s: out_dtype %d", fn, out_dtype);
  TRY(check_shape(fn, 16, first, E, R, N, K));
  TRY(check_rows(fn, rows, x_rows, R));
  if (K > kI8MaxK) return fail(MOE_EUNSUPPORTED, "%s: K=%d above %d (32-bit sums)", fn, K, kI8MaxK);
  if (!first && E != 1) return fail(MOE_EINVAL, "%s: null first", fn);
  if (R == 0) return MOE_OK;
  const void *p[] = {w, out, x};   // an x without rows is not read
  TRY(check_ptrs(fn, p, x_rows ? 3 : 2));
  if ((!x_scales && x_rows) || !w_scales || !aligned(x_scales, 4) || !aligned(w_scales, 4))
    return fail(MOE_EINVAL, "%s: null or misaligned scales", fn);
  Span work;
  TRY(check_scratch(fn, MOE_MM_INT8, E, R, N, K, scratch, scratch_bytes, &work));
  TRY(check_apart(fn, {{out, (size_t)R * N * type_size(out_dtype)}, work},
                  {{x, (size_t)x_rows * K}, {x_scales, x_rows * sizeof *x_scales}, {w, (size_t)E * N * K},
                   {w_scales, (size_t)E * N * sizeof *w_scales}, {first, (E + 1) * sizeof *first},
                   {rows, R * sizeof *rows}}));
  moe::MmArgs a = {};
  a.part = (float *)scratch;
  a.op = moe::MM_FORWARD, a.type = moe::MM_I8, a.out_type = out_dtype;
  a.x = x, a.x_rows = (long)x_rows, a.rows = rows, a.x_scales = x_scales, a.w = w, a.w_scales = w_scales;
  a.first = first, a.E = E, a.R = R, a.N = N, a.K = K, a.out = out;
  return launched(moe::launch_mm(a, (hipStream_t)stream), fn);
}

int moe_int8_mm(const int8_t *x, const float *x_scales, const int8_t *w, const float *w_scales, int M, int N, int K,
                int out_dtype, void *out, void *scratch, size_t scratch_bytes, void *stream) {
  return moe_grouped_int8_mm(x, x_scales, M, nullptr, w, w_scales, nullptr, 1, M, N, K, out_dtype, out, scratch,
                             scratch_bytes, stream);
}

size_t moe_group_routes_scratch_bytes(int T, int top_k, int E) {
  if (T < 0 || top_k < 1 || E < 1 || (long long)T * top_k > INT32_MAX) return 0;
  const long R = (long)T * top_k;
  return R <= 4 * moe::kGroupThreads ? 0 : sizeof(int32_t) * ((size_t)moe::group_blocks(R) * E + R);
}

int moe_group_routes(const int32_t *topk_ids, int T, int top_k, int E, int32_t *first, int32_t *order, int32_t *token,
                     int32_t *inverse, void *scratch, size_t scratch_bytes, void *stream) {
  const char *fn = "moe_group_routes";
  if (T < 0 || E < 1) return fail(MOE_EINVAL, "%s: T=%d, E=%d", fn, T, E);
  if (top_k < 1 || top_k > 64) return fail(MOE_EINVAL, "%s: top_k=%d outside [1, 64]", fn, top_k);
  if (E > moe::kMaxExperts) return fail(MOE_EUNSUPPORTED, "%s: E=%d above %d", fn, E, moe::kMaxExperts);
  if ((long long)T * top_k > (1 << 30)) return fail(MOE_EUNSUPPORTED, "%s: more than 2^30 routes", fn);
  const void *p[] = {first, topk_ids, order, token, inverse};   // without routes only first is written
  for (int i = 0; i < (T ? 5 : 1); i++)
    if (!p[i] || !aligned(p[i], 4)) return fail(MOE_EINVAL, "%s: null or misaligned pointer (4 bytes)", fn);
  const size_t need = moe_group_routes_scratch_bytes(T, top_k, E);
  if (need && (!scratch || !aligned(scratch, 4))) return fail(MOE_EINVAL, "%s: null or misaligned scratch", fn);
  if (scratch_bytes < need) return fail(MOE_ESCRATCH, "%s: scratch holds %zu bytes, %zu needed", fn, scratch_bytes, need);
  const size_t ids_bytes = (size_t)T * top_k * sizeof *topk_ids;
  TRY(check_apart(fn, {{first, (E + 1) * sizeof *first}, {order, ids_bytes}, {token, ids_bytes}, {inverse, ids_bytes},
                       {need ? scratch : nullptr, need}}, {{topk_ids, ids_bytes}}));
  moe::GroupArgs a = {};
  a.ids = topk_ids, a.R = T * top_k, a.topk = top_k, a.E = E;
  if (need) a.rounds = moe::group_rounds(a.R), a.blocks = moe::group_blocks(a.R);
  a.first = first, a.order = order, a.token = token, a.inverse = inverse;
  a.hist = (int32_t *)scratch, a.rank = (int32_t *)scratch + (size_t)a.blocks * E;
  return launched(moe::launch_group(a, (hipStream_t)stream), fn);
}

}  // extern "C"
