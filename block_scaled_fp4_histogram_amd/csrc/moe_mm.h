// Internal declarations of the ragged expert products, the 8-bit integer
// products, the row quantiser and the route grouping (moe_mm.hip, moe_rows.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

enum MmType { MM_BF16 = 1, MM_FP16 = 2, MM_FP32 = 3, MM_I8 = 4 };
enum MmOp { MM_FORWARD = 1, MM_DX = 2, MM_DW = 3 };

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
  const float *x_scales, *w_scales;  // MM_I8: per row of x, per channel [E, N]
  void *out;                         // [R, N], [R, K] or [E, N, K]
  float *part;                       // scratch of a split reduction: [splits] of out in 32 bits
  int splits;                        // set by launch_mm
};

// How a product of these sizes runs: by streaming or in tiles of a shape, with
// the reduction in how many parts, and the scratch bytes those take.  Host only,
// from the sizes alone.
struct MmPlan {
  int stream, shape, splits;
  int rows, cols;                    // of a tile
  size_t scratch;
};
MmPlan mm_plan(int op, int type, long E, long R, long N, long K);

hipError_t launch_mm(const MmArgs &a, hipStream_t s);

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
