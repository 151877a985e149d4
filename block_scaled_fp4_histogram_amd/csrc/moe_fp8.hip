// Products over 8-bit floating point (E4M3) with a scale for each block of 128 for
// gfx950, alone and as a gated block, and the quantiser of their rows.
#include <algorithm>

#include "moe_mm_tile.h"

namespace moe {

// One group of 16384 x 4096 x 4096, summed in fp32: 537, 497, 550, 586 us (1.11 PFLOP/s; the
// conversions and scales issue about as long as the matrix cores are busy).
template <int OP>
static hipError_t launch_fp8_tiles(const MmArgs &a, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_tile<OP, MM_F8X, 256, 128, 4, 1, 2>(a, s);
    case 1: return launch_tile<OP, MM_F8X, 128, 256, 2, 2, 2>(a, s);
    case 2: return launch_tile<OP, MM_F8X, 128, 128, 2, 2, 2>(a, s);
    default: return launch_tile<OP, MM_F8X, 64, 128, 2, 2, 4>(a, s);
  }
}

// By the 8-bit instruction: 313, 295, 312, 356 us, repeated 271 (2.0 PFLOP/s; with two waves a SIMD the
// loads' and the scales' waits stand between the products).
template <int OP>
static hipError_t launch_fp8_fast(const MmArgs &a, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_tile<OP, MM_F8, 256, 128, 4, 1, 2>(a, s);
    case 1: return launch_tile<OP, MM_F8, 128, 256, 2, 2, 2>(a, s);
    case 2: return launch_tile<OP, MM_F8, 128, 128, 2, 2, 3>(a, s);
    default: return launch_tile<OP, MM_F8, 64, 128, 2, 2, 4>(a, s);
  }
}

template <int OP>
static hipError_t launch_fp8_op(const MmArgs &a, const MmPlan &m, hipStream_t s) {
  if (m.stream) return launch_stream<OP, MM_F8X>(a, s);
  return a.type == MM_F8 ? launch_fp8_fast<OP>(a, m.shape, s) : launch_fp8_tiles<OP>(a, m.shape, s);
}

hipError_t launch_fp8(const MmArgs &a, const MmPlan &m, hipStream_t s) {
  return a.op == MM_GLU ? launch_fp8_op<MM_GLU>(a, m, s) : launch_fp8_op<MM_FORWARD>(a, m, s);
}

// ------------------------------------------------------------ quantiser

// Sixteen lanes a block of 128 columns, eight values a lane: the block's largest
// magnitude by its bits (which order as the values do, infinities and NaN above
// all), then the codes of x * fp32(448 / amax).  Blocks too small for that factor
// to stay in range are worked 2^64 larger, which is exact.  A block that holds an
// infinity or NaN gets scale NaN and codes 0, so its products are NaN.  CH blocks a
// turn, whose loads are in flight together.
template <int TYPE, int CH>
__global__ __launch_bounds__(256) void k_quant_fp8(const uint16_t *x, long units, int kbs, int cols, uint8_t *q, float *scales) {
  typedef uint16_t v2us __attribute__((ext_vector_type(2)));
  const int l = threadIdx.x & 15;
  for (long u0 = ((long)blockIdx.x * 16 + (threadIdx.x >> 4)) * CH; u0 < units; u0 += (long)gridDim.x * 16 * CH) {
    v4i v[CH];
    long at[CH];                         // first of the lane's values (-1: none)
#pragma unroll
    for (int i = 0; i < CH; i++) {
      const long row = (u0 + i) / kbs;
      const int c = (int)(u0 + i - row * kbs) * 128 + l * 8;
      at[i] = u0 + i < units && c < cols ? row * cols + c : -1;
      v[i] = at[i] < 0 ? v4i{0, 0, 0, 0} : *(const v4i *)(x + at[i]);
    }
#pragma unroll
    for (int i = 0; i < CH; i++) {
      v2us mm = {0, 0};
#pragma unroll
      for (int d = 0; d < 4; d++) mm = __builtin_elementwise_max(mm, __builtin_bit_cast(v2us, (uint32_t)v[i][d] & 0x7FFF7FFFu));
      const uint32_t m = row16_max(max((uint32_t)mm[0], (uint32_t)mm[1]));
      const bool bad = m >= (TYPE == MM_BF16 ? 0x7F80u : 0x7C00u);
      const float amax = glu_elem<TYPE>(m, 0), up = amax < 0x1p-100f ? 0x1p64f : 1.0f;
      const float r = m == 0 || bad ? 0.0f : 448.0f / (amax * up);
      if (l == 0 && u0 + i < units) scales[u0 + i] = bad ? __uint_as_float(0x7FC00000u) : amax / 448.0f;
      uint32_t o[2];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; k++) f[k] = glu_elem<TYPE>(v[i][2 * h + (k >> 1)], k & 1) * up * r;
        o[h] = e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16;
      }
      if (at[i] >= 0) *(v2u *)(q + at[i]) = bad ? v2u{0, 0} : v2u{o[0], o[1]};
    }
  }
}

// Two blocks a turn from 2^17 of them on (16384 rows of 4096: 40.0 us with one, 37.8 with
// two, 37.1 with four; 4097 of 7168: 20.2, 18.8, 19.1, 4.7 TB/s), one below, where more
// waves are worth more than loads in flight (512 rows of 7168: 4.0, 4.4, 4.8 us).
template <int TYPE>
static hipError_t launch_quant(const uint16_t *x, long units, int kbs, int cols, uint8_t *q, float *scales, hipStream_t s) {
  const int ch = units >= 1l << 17 ? 2 : 1;
  const dim3 grid((unsigned)std::min((units + 16 * ch - 1) / (16 * ch), 1l << 20)), threads(256);
  if (ch == 2) hipLaunchKernelGGL((k_quant_fp8<TYPE, 2>), grid, threads, 0, s, x, units, kbs, cols, q, scales);
  else hipLaunchKernelGGL((k_quant_fp8<TYPE, 1>), grid, threads, 0, s, x, units, kbs, cols, q, scales);
  return hipGetLastError();
}

hipError_t launch_quant_fp8(int type, const void *x, long rows, int cols, uint8_t *q, float *scales, hipStream_t s) {
  const int kbs = (cols + kF8Block - 1) / kF8Block;
  return type == MM_BF16 ? launch_quant<MM_BF16>((const uint16_t *)x, rows * kbs, kbs, cols, q, scales, s)
                         : launch_quant<MM_FP16>((const uint16_t *)x, rows * kbs, kbs, cols, q, scales, s);
}

}  // namespace moe
