// Internal declarations of the ragged expert products, the 8-bit integer and
// floating-point products, the gated block, the row quantisers and the route
// grouping (moe_mm.hip, moe_glu.hip, moe_fp8.hip, moe_rows.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

enum MmType { MM_BF16 = 1, MM_FP16 = 2, MM_FP32 = 3, MM_I8 = 4, MM_F8 = 5, MM_F8X = 6 };
// (MM_F8X: the same operands as MM_F8, summed in fp32 in place of by the 8-bit matrix
// instruction, which the caller asks for.)
// MM_GLU: a forward product with the gate's and the up branch's rows of w, N of each,
// then the activation; MM_GLU_DX: MM_DX, then the activation's gradient.
enum MmOp { MM_FORWARD = 1, MM_DX = 2, MM_DW = 3, MM_GLU = 4, MM_GLU_DX = 5 };

// The activation of a gated block of I columns, and where its branches lie in rows
// (of w) or columns (of the projections) of 2 I: gate0 and up0 are 0 and I or I and 0.
struct GluForm {
  int act, has_limit;
  float limit, alpha, beta;
  int gate0, up0;
};

// One product over E groups of rows; group e holds rows first[e] .. first[e+1]
// (first == NULL: one group of R rows).  Every kernel clamps the offsets to
// [0, R], so no offset array makes it leave its buffers.
struct MmArgs {
  int op, type, out_type, accumulate;
  const void *x;                     // MM_FORWARD, MM_DW: rows of K
  const void *dy;                    // MM_DX, MM_DW: rows of N
  const void *w;                     // MM_FORWARD, MM_DX: [E, N, K]
  const int32_t *rows;               // row of x behind each product row (NULL: its own)
  long x_rows;                       // rows of x (checked against `rows` on the device)
  const int32_t *first;
  int E, R, N, K;
  const float *x_scales, *w_scales;  // MM_I8: per row of x, per channel [E, N]; MM_F8 and MM_F8X: per block of 128
  void *out;                         // [R, N], [R, K] or [E, N, K]; MM_GLU_DX: the projections' gradient [R, 2 K]
  float *part;                       // scratch of a split reduction: [splits] of out in 32 bits
  int splits;                        // set by launch_mm
  int tail;                          // set by launch_mm: the last round's tiles are split (mm_tail)
  GluForm glu;                       // MM_GLU, MM_GLU_DX
  const void *pre;                   // MM_GLU_DX: the projections [R, 2 K]
  void *pre_out;                     // MM_GLU: the projections [R, 2 N], or NULL
  void *h;                           // MM_GLU_DX: the activation [R, K], or NULL
};

// How a product of these sizes runs: by streaming or in tiles of a shape, with
// the reduction in how many parts, and the scratch bytes those take.  Host only,
// from the sizes alone.
struct MmPlan {
  int stream, shape, splits;
  int rows, cols;                    // of a tile
  int tail;                          // the tiles of the last round in parts
  size_t scratch;
};
MmPlan mm_plan(int op, int type, long E, long R, long N, long K);

hipError_t launch_mm(const MmArgs &a, hipStream_t s);
// The same for MM_GLU and MM_GLU_DX of 16-bit operands, and for MM_F8 and MM_F8X, under plan m.
hipError_t launch_glu(const MmArgs &a, const MmPlan &m, hipStream_t s);
hipError_t launch_fp8(const MmArgs &a, const MmPlan &m, hipStream_t s);

// The activation's gradient from dh [R, I] alone.
hipError_t launch_glu_grad(int type, const void *dh, const void *pre, long R, int I, const GluForm &f, void *d_pre,
                           void *h, hipStream_t s);

// Quantiser to E4M3: blocks of 128 columns of a row, scale = fp32(amax / 448).
hipError_t launch_quant_fp8(int type, const void *x, long rows, int cols, uint8_t *q, float *scales, hipStream_t s);

// Row quantiser: scale = fp32(amax / 127), codes = x / scale to nearest even.
hipError_t launch_quant_int8(int type, const void *x, long rows, int cols, int8_t *q, float *scales, hipStream_t s);

constexpr int kGroupThreads = 1024;  // routes a block of the grouping kernels takes a round
constexpr int kGroupFew = 256;       // most routes of the kernel without counting
constexpr int kGroupMaxBlocks = 256; // most blocks of the counting kernels; more routes take more rounds

struct GroupArgs {
  const int32_t *ids;
  int R, topk, E;
  int blocks, rounds;                // of the two-launch form (R > 4 * kGroupThreads)
  int32_t *first, *order, *token, *inverse;
  int32_t *hist, *rank;              // its scratch: [blocks][E] counts, per-route rank
};

// Blocks and rounds of R routes in the two-launch form.
constexpr int group_rounds(long R) {
  return (int)((R + (long)kGroupThreads * kGroupMaxBlocks - 1) / ((long)kGroupThreads * kGroupMaxBlocks));
}
constexpr int group_blocks(long R) {
  return (int)((R + (long)kGroupThreads * group_rounds(R) - 1) / ((long)kGroupThreads * group_rounds(R)));
}

hipError_t launch_group(const GroupArgs &a, hipStream_t s);

}  // namespace moe
