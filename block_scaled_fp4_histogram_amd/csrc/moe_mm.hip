// Ragged expert products for gfx950: forward, row gradient and weight gradient
// over 16-bit operands, and the forward product over 8-bit integers.
#include "moe_device.h"
#include "moe_mm.h"

namespace moe {

// Group, first row and row count of row tile `tile` (tiles of BM rows, groups
// in order); rows == 0 when the groups hold fewer tiles.  One wave reads 64
// offsets at a time and scans their tile counts; every wave of a block does
// the same work, so no barrier is needed.
struct MmTile {
  int e, row0, rows;
};

template <int BM>
__device__ MmTile mm_tile(const MmArgs &a, int tile) {
  MmTile t = {0, 0, 0};
  if (!a.first) {
    t.row0 = tile * BM;
    t.rows = min(BM, a.R - t.row0);
    return t;
  }
  const int lane = threadIdx.x & 63;
  int run = 0;
  for (int b = 0; b < a.E; b += 64) {
    const int e = b + lane;
    int lo = 0, hi = 0;
    if (e < a.E) {
      lo = min(max(a.first[e], 0), a.R);
      hi = min(max(a.first[e + 1], lo), a.R);
    }
    const int c = (hi - lo + BM - 1) / BM;
    int s = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(s, d);
      if (lane >= d) s += v;
    }
    const int total = __shfl(s, 63);
    if (tile < run + total) {
      const unsigned long long m = __ballot(run + s > tile);
      const int src = __ffsll(m) - 1;
      const int before = run + __shfl(s - c, src);
      t.e = b + src;
      t.row0 = __shfl(lo, src) + (tile - before) * BM;
      t.rows = max(0, min(BM, __shfl(hi, src) - t.row0));
      return t;
    }
    run += total;
  }
  return t;
}

template <int TYPE>
struct MmElem;
template <>
struct MmElem<MM_BF16> {
  typedef uint16_t t;
  typedef v4f acc;
  static __device__ __forceinline__ v4f mma(v4i p, v4i q, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, p), __builtin_bit_cast(v8bf, q), c, 0, 0, 0);
  }
};
template <>
struct MmElem<MM_FP16> {
  typedef uint16_t t;
  typedef v4f acc;
  static __device__ __forceinline__ v4f mma(v4i p, v4i q, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, p), __builtin_bit_cast(v8h, q), c, 0, 0, 0);
  }
};
template <>
struct MmElem<MM_I8> {
  typedef uint8_t t;
  typedef v4i acc;
  static __device__ __forceinline__ v4i mma(v4i p, v4i q, v4i c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(p, q, c, 0, 0, 0);
  }
};

__device__ __forceinline__ void mm_store(const MmArgs &a, long at, float v) {
  if (a.out_type == MM_FP32) {
    float *o = (float *)a.out + at;
    *o = a.accumulate ? *o + v : v;
  } else if (a.out_type == MM_BF16) {
    ((uint16_t *)a.out)[at] = (uint16_t)pack_bf16x2(v, 0.f);
  } else {
    ((_Float16 *)a.out)[at] = (_Float16)v;
  }
}

// 64 x 64 output tile per block of four waves (32 x 32 each, 16 x 16 MFMAs),
// operands staged in LDS with the reduction contiguous.  P holds the output's
// contiguous side, Q its rows.
template <int OP, int TYPE>
__global__ __launch_bounds__(256) void k_mm(MmArgs a) {
  typedef MmElem<TYPE> M;
  typedef typename M::t T;
  constexpr int ZB = 64 / sizeof(T);        // reduction elements per step: 64 bytes
  constexpr int C = 16 / sizeof(T);         // elements per 16-byte chunk
  __shared__ __align__(16) T lp[64][ZB + C], lq[64][ZB + C];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  MmTile t;
  int q0, qn, p0 = (int)blockIdx.x * 64, pn, zn;
  if (OP == MM_DW) {
    t.e = blockIdx.z;
    const int lo = min(max(a.first ? a.first[t.e] : 0, 0), a.R);
    t.row0 = lo;
    t.rows = (a.first ? min(max(a.first[t.e + 1], lo), a.R) : a.R) - lo;
    q0 = blockIdx.y * 64;
    qn = a.N;
    pn = a.K;
    zn = t.rows;
  } else {
    t = mm_tile<64>(a, blockIdx.y);
    if (t.rows <= 0) return;
    q0 = 0;
    qn = t.rows;
    pn = OP == MM_FORWARD ? a.N : a.K;
    zn = OP == MM_FORWARD ? a.K : a.N;
  }
  const T *x = (const T *)a.x, *dy = (const T *)a.dy, *wt = (const T *)a.w + (long)t.e * a.N * a.K;
  // 16 bytes of row i of x behind product row r, zeros where there is none
  auto x_chunk = [&](int r, int col) -> v4i {
    long xr = r;
    if (a.rows) {
      xr = a.rows[r];
      if (xr < 0 || xr >= a.x_rows) return v4i{0, 0, 0, 0};
    }
    return *(const v4i *)(x + xr * a.K + col);
  };
  typename M::acc acc[2][2] = {};
  for (int z0 = 0; z0 < zn; z0 += ZB) {
    __syncthreads();
    // Q
    if (OP != MM_DW) {
      const int row = tid >> 2, col = z0 + (tid & 3) * C;
      v4i v = {0, 0, 0, 0};
      if (row < qn && col < zn)
        v = OP == MM_FORWARD ? x_chunk(t.row0 + row, col) : *(const v4i *)(dy + (long)(t.row0 + row) * a.N + col);
      *(v4i *)&lq[row][(tid & 3) * C] = v;
    } else {
      const int z = tid >> 3, col = q0 + (tid & 7) * 8;
      v4i v = {0, 0, 0, 0};
      if (z0 + z < zn && col < qn) v = *(const v4i *)(dy + (long)(t.row0 + z0 + z) * a.N + col);
      for (int i = 0; i < 8; i++) lq[(tid & 7) * 8 + i][z] = (T)((uint32_t)v[i >> 1] >> (16 * (i & 1)));
    }
    // P
    if (OP == MM_FORWARD) {
      const int row = p0 + (tid >> 2), col = z0 + (tid & 3) * C;
      v4i v = {0, 0, 0, 0};
      if (row < pn && col < zn) v = *(const v4i *)(wt + (long)row * a.K + col);
      *(v4i *)&lp[tid >> 2][(tid & 3) * C] = v;
    } else {
      const int z = tid >> 3, col = p0 + (tid & 7) * 8;
      v4i v = {0, 0, 0, 0};
      if (z0 + z < zn && col < pn)
        v = OP == MM_DX ? *(const v4i *)(wt + (long)(z0 + z) * a.K + col) : x_chunk(t.row0 + z0 + z, col);
      for (int i = 0; i < 8; i++) lp[(tid & 7) * 8 + i][z] = (T)((uint32_t)v[i >> 1] >> (16 * (i & 1)));
    }
    __syncthreads();
    v4i fp[2], fq[2];
    for (int i = 0; i < 2; i++) {
      fp[i] = *(const v4i *)&lp[32 * (w & 1) + 16 * i + (lane & 15)][(lane >> 4) * C];
      fq[i] = *(const v4i *)&lq[32 * (w >> 1) + 16 * i + (lane & 15)][(lane >> 4) * C];
    }
    for (int i = 0; i < 2; i++)
      for (int j = 0; j < 2; j++) acc[i][j] = M::mma(fp[i], fq[j], acc[i][j]);
  }
  for (int i = 0; i < 2; i++)
    for (int j = 0; j < 2; j++) {
      const int q = q0 + 32 * (w >> 1) + 16 * j + (lane & 15), p = p0 + 32 * (w & 1) + 16 * i + 4 * (lane >> 4);
      if (q >= qn) continue;
      const long row = OP == MM_DW ? (long)t.e * a.N + q : t.row0 + q;
      for (int k = 0; k < 4; k++) {
        if (p + k >= pn) continue;
        float v = (float)acc[i][j][k];
        if (TYPE == MM_I8) {
          long xr = row;
          if (a.rows) {
            xr = a.rows[row];
            if (xr < 0 || xr >= a.x_rows) xr = -1;
          }
          v = xr < 0 ? 0.f : v * a.x_scales[xr] * a.w_scales[(long)t.e * a.N + p + k];
        }
        mm_store(a, row * pn + p + k, v);
      }
    }
}

template <int OP, int TYPE>
static hipError_t launch_mm_simple(const MmArgs &a, hipStream_t s) {
  const int pn = OP == MM_FORWARD ? a.N : a.K;
  const int tiles = a.first ? (a.R + 63) / 64 + (a.E < a.R ? a.E : a.R) : (a.R + 63) / 64;
  const dim3 grid((pn + 63) / 64, OP == MM_DW ? (a.N + 63) / 64 : tiles, OP == MM_DW ? a.E : 1);
  hipLaunchKernelGGL((k_mm<OP, TYPE>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_mm(const MmArgs &a, hipStream_t s) {
  if (a.type == MM_I8) return launch_mm_simple<MM_FORWARD, MM_I8>(a, s);
  if (a.type == MM_BF16)
    return a.op == MM_FORWARD ? launch_mm_simple<MM_FORWARD, MM_BF16>(a, s)
           : a.op == MM_DX    ? launch_mm_simple<MM_DX, MM_BF16>(a, s)
                              : launch_mm_simple<MM_DW, MM_BF16>(a, s);
  return a.op == MM_FORWARD ? launch_mm_simple<MM_FORWARD, MM_FP16>(a, s)
         : a.op == MM_DX    ? launch_mm_simple<MM_DX, MM_FP16>(a, s)
                            : launch_mm_simple<MM_DW, MM_FP16>(a, s);
}

}  // namespace moe
