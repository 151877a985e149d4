// Row kernels next to the products, for gfx950: the 8-bit integer quantiser
// and the grouping of routes by expert.
#include "moe_device.h"
#include "moe_mm.h"

namespace moe {

// ------------------------------------------------------------ quantiser

template <int TYPE>
__device__ __forceinline__ float row_elem(uint32_t d, int h) {
  const uint32_t u = (h ? d >> 16 : d & 0xFFFFu);
  return TYPE == MM_BF16 ? bf16_to_f32(u) : (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}

// The integer nearest to x / s (ties to even) for |x| <= 127.5 s: the fp32
// product r = x * inv is within one of it; the remainder x - rint(r) s is a
// multiple of s's last place (or of x's, if that is finer) below 2^25 of them,
// so the fma gives it exactly and its comparison with s / 2 decides.
__device__ __forceinline__ int quant_code(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float e = 2.0f * fmaf(-q, s, x);
  if (e > s || (e == s && ((int)q & 1))) q += 1.0f;
  else if (e < -s || (e == -s && ((int)q & 1))) q -= 1.0f;
  return (int)__builtin_amdgcn_fmed3f(q, -127.0f, 127.0f);
}

// One block per row: the row's largest magnitude, then its codes.  A row with
// an infinity or NaN gets scale NaN and codes 0, so its products are NaN.
template <int TYPE>
__global__ __launch_bounds__(256) void k_quant_int8(const uint16_t *x, int cols, int8_t *q, float *scales) {
  __shared__ uint32_t red[4];
  const long row = blockIdx.x;
  const v4i *src = (const v4i *)(x + row * cols);
  const int n = cols / 8;
  uint32_t m = 0;
  for (int i = threadIdx.x; i < n; i += 256) {
    const v4i v = src[i];
#pragma unroll
    for (int d = 0; d < 4; d++) m = max(m, max((uint32_t)v[d] & 0x7FFFu, ((uint32_t)v[d] >> 16) & 0x7FFFu));
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  const bool bad = m >= (TYPE == MM_BF16 ? 0x7F80u : 0x7C00u);
  const float amax = row_elem<TYPE>(m, 0);
  const float s = bad ? __uint_as_float(0x7FC00000u) : amax / 127.0f;
  if (threadIdx.x == 0) scales[row] = s;
  const bool zero = bad || s == 0.0f;
  // rows too small for 127 / amax to stay in range are worked 2^64 larger (exact)
  const float up = amax < 1e-30f ? 0x1p64f : 1.0f;
  const float su = s * up, inv = zero ? 0.0f : 127.0f / (amax * up);
  for (int i = threadIdx.x; i < n; i += 256) {
    const v4i v = src[i];
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float f = row_elem<TYPE>((uint32_t)v[j >> 1], j & 1) * up;
      const int c = zero ? 0 : quant_code(f, su, inv);
      o[j >> 2] |= ((uint32_t)c & 0xFFu) << (8 * (j & 3));
    }
    typedef uint32_t v2u __attribute__((ext_vector_type(2)));
    ((v2u *)(q + row * cols))[i] = v2u{o[0], o[1]};
  }
}

hipError_t launch_quant_int8(int type, const void *x, long rows, int cols, int8_t *q, float *scales, hipStream_t s) {
  if (type == MM_BF16)
    hipLaunchKernelGGL(k_quant_int8<MM_BF16>, dim3((unsigned)rows), dim3(256), 0, s, (const uint16_t *)x, cols, q, scales);
  else
    hipLaunchKernelGGL(k_quant_int8<MM_FP16>, dim3((unsigned)rows), dim3(256), 0, s, (const uint16_t *)x, cols, q, scales);
  return hipGetLastError();
}

// ------------------------------------------------------------ grouping

constexpr int kGroupMaxE = 1024;
constexpr int kGroupWaves = kGroupChunk / 64;

// Exclusive prefix of cnt[0 .. E) into off[0 .. E], by the block's first wave.
__device__ void group_offsets(int E, const int *cnt, int *off) {
  const int lane = threadIdx.x;
  if (lane < 64) {
    const int per = (E + 63) / 64, b = lane * per;
    int s = 0;
    for (int i = b; i < min(b + per, E); i++) s += cnt[i];
    int inc = s;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(inc, d);
      if (lane >= d) inc += v;
    }
    int run = inc - s;
    for (int i = b; i < min(b + per, E); i++) {
      off[i] = run;
      run += cnt[i];
    }
    if (lane == 63) off[E] = inc;
  }
}

__device__ __forceinline__ void group_place(const GroupArgs &a, int r, int e, int pos) {
  a.inverse[r] = e < 0 ? -1 : pos;
  if (e >= 0) {
    a.order[pos] = r;
    a.token[pos] = r / a.topk;
  }
}

// Counting sort, one route per thread: its rank among the routes of the same
// expert before it, first within its wave (the lanes of one expert are found
// together by ballots), then over the chunk's waves.  ONE: a single chunk,
// offsets and placement in the same launch; otherwise the chunk's counts and
// the ranks go to scratch.
template <bool ONE>
__global__ __launch_bounds__(kGroupChunk) void k_group(GroupArgs a) {
  __shared__ uint16_t whist[kGroupWaves][kGroupMaxE];
  __shared__ int cnt[kGroupMaxE], off[kGroupMaxE + 1];
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  for (int i = tid; i < kGroupWaves * a.E; i += kGroupChunk) whist[i / a.E][i % a.E] = 0;
  __syncthreads();
  const int r = blockIdx.x * kGroupChunk + tid;
  int e = r < a.R ? a.ids[r] : -1;
  if (e < 0 || e >= a.E) e = -1;
  int rank = 0;
  unsigned long long rem = __ballot(e >= 0);
  while (rem) {
    const int leader = __ffsll(rem) - 1;
    const int le = __shfl(e, leader);
    const unsigned long long m = __ballot(e == le);
    if (e == le) rank = __popcll(m & ((1ull << lane) - 1ull));
    if (lane == leader) whist[w][le] = (uint16_t)__popcll(m);
    rem &= ~m;
  }
  __syncthreads();
  for (int i = tid; i < a.E; i += kGroupChunk) {
    int run = 0;
#pragma unroll
    for (int v = 0; v < kGroupWaves; v++) {
      const int c = whist[v][i];
      whist[v][i] = (uint16_t)run;
      run += c;
    }
    if (ONE) cnt[i] = run;
    else a.hist[(long)blockIdx.x * a.E + i] = run;
  }
  __syncthreads();
  if (e >= 0) rank += whist[w][e];
  if (!ONE) {
    if (r < a.R) a.rank[r] = rank;
    return;
  }
  group_offsets(a.E, cnt, off);
  __syncthreads();
  for (int i = tid; i <= a.E; i += kGroupChunk) a.first[i] = off[i];
  if (r < a.R) {
    group_place(a, r, e, e < 0 ? 0 : off[e] + rank);
    if (r >= off[a.E]) a.order[r] = a.token[r] = -1;
  }
}

// Placement of one chunk: each block sums the chunks' counts itself (all of
// them, and those before its own), which saves a launch for the scan.
__global__ __launch_bounds__(kGroupChunk) void k_group_place(GroupArgs a) {
  __shared__ int cnt[kGroupMaxE], before[kGroupMaxE], off[kGroupMaxE + 1];
  const int tid = threadIdx.x;
  for (int i = tid; i < a.E; i += kGroupChunk) {
    int run = 0, mine = 0;
    for (int c = 0; c < a.chunks; c++) {
      if (c == (int)blockIdx.x) mine = run;
      run += a.hist[(long)c * a.E + i];
    }
    cnt[i] = run;
    before[i] = mine;
  }
  __syncthreads();
  group_offsets(a.E, cnt, off);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = tid; i <= a.E; i += kGroupChunk) a.first[i] = off[i];
  const int r = blockIdx.x * kGroupChunk + tid;
  if (r >= a.R) return;
  int e = a.ids[r];
  if (e < 0 || e >= a.E) e = -1;
  group_place(a, r, e, e < 0 ? 0 : off[e] + before[e] + a.rank[r]);
  if (r >= off[a.E]) a.order[r] = a.token[r] = -1;
}

hipError_t launch_group(const GroupArgs &a, hipStream_t s) {
  if (a.chunks <= 1) {
    hipLaunchKernelGGL(k_group<true>, dim3(1), dim3(kGroupChunk), 0, s, a);
  } else {
    hipLaunchKernelGGL(k_group<false>, dim3(a.chunks), dim3(kGroupChunk), 0, s, a);
    hipLaunchKernelGGL(k_group_place, dim3(a.chunks), dim3(kGroupChunk), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
