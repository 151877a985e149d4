// The gated feed-forward block on 16-bit operands for gfx950: both projections and
// the activation in one product, and the backward pass through the activation.
#include "moe_mm_tile.h"

namespace moe {

// Tiles of the products' shapes, whose waves here hold as many columns of each
// branch; 256 x 128 with all four waves over the rows, so that a wave's rows of h are whole
// lines (64 columns in 16 bits).  16384 x 2 x 2048 x 4096, bf16: 425, 420, 452, 555 us
// (1.29 PFLOP/s); bound by the matrix cores and the clock they leave.
template <int TYPE>
static hipError_t launch_glu_tiles(const MmArgs &a, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_tile<MM_GLU, TYPE, 256, 128, 4, 1, 2>(a, s);
    case 1: return launch_tile<MM_GLU, TYPE, 128, 256, 2, 2, 2>(a, s);
    case 2: return launch_tile<MM_GLU, TYPE, 128, 128, 2, 2, 3>(a, s);
    default: return launch_tile<MM_GLU, TYPE, 64, 128, 2, 2, 4>(a, s);
  }
}

// Row gradients with the activation's gradient behind them.  32 groups of 512 rows, 6144 x
// 1024, h once more: 228, 235, 296, 324 us, the row gradient alone 207, 203, 263, 302; the
// epilogue's 10 bytes an output are read and written when the products of its round end.
template <int TYPE>
static hipError_t launch_glu_dx(const MmArgs &a, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_tile<MM_GLU_DX, TYPE, 256, 128, 2, 2, 2>(a, s);
    case 1: return launch_tile<MM_GLU_DX, TYPE, 128, 256, 2, 2, 2>(a, s);
    case 2: return launch_tile<MM_GLU_DX, TYPE, 128, 128, 2, 2, 3>(a, s);
    default: return launch_tile<MM_GLU_DX, TYPE, 64, 128, 2, 2, 4>(a, s);
  }
}

template <int TYPE>
static hipError_t launch_glu_type(const MmArgs &a, const MmPlan &m, hipStream_t s) {
  if (a.op == MM_GLU_DX) return launch_glu_dx<TYPE>(a, m.shape, s);
  return m.stream ? launch_stream<MM_GLU, TYPE>(a, s) : launch_glu_tiles<TYPE>(a, m.shape, s);
}

hipError_t launch_glu(const MmArgs &a, const MmPlan &m, hipStream_t s) {
  return a.type == MM_BF16 ? launch_glu_type<MM_BF16>(a, m, s) : launch_glu_type<MM_FP16>(a, m, s);
}

// The gradient where dh is in memory: a pass over it, eight columns a thread (16382 x 2048
// with h once more, 0.4 GB: 70 us, 5.8 TB/s; bound by HBM).
template <int TYPE>
__global__ __launch_bounds__(256) void k_glu_grad(const uint16_t *dh, const void *pre, long chunks, int I, GluForm f,
                                                  void *d_pre, void *h) {
  const int per = I / 8;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (long)gridDim.x * 256) {
    const long r = i / per;
    const int c = (int)(i - r * per) * 8;
    const v4i v = *(const v4i *)(dh + i * 8);
    v4f d[2];
#pragma unroll
    for (int k = 0; k < 8; k++) d[k >> 2][k & 3] = glu_elem<TYPE>(v[k >> 1], k & 1);
    glu_back8<TYPE>(f, I, pre, d_pre, h, r, c, d[0], d[1]);
  }
}

hipError_t launch_glu_grad(int type, const void *dh, const void *pre, long R, int I, const GluForm &f, void *d_pre,
                           void *h, hipStream_t s) {
  const long chunks = R * (I / 8), blocks = (chunks + 255) / 256;
  const dim3 grid((unsigned)(blocks < 1l << 20 ? blocks : 1l << 20)), threads(256);
  if (type == MM_BF16) hipLaunchKernelGGL(k_glu_grad<MM_BF16>, grid, threads, 0, s, (const uint16_t *)dh, pre, chunks, I, f, d_pre, h);
  else hipLaunchKernelGGL(k_glu_grad<MM_FP16>, grid, threads, 0, s, (const uint16_t *)dh, pre, chunks, I, f, d_pre, h);
  return hipGetLastError();
}

}  // namespace moe
