// Row kernels next to the products, for gfx950: the 8-bit integer quantiser
// and the grouping of routes by expert.
#include <algorithm>

#include "moe_device.h"
#include "moe_mm.h"

namespace moe {

// ------------------------------------------------------------ quantiser

template <int TYPE>
__device__ __forceinline__ float row_elem(uint32_t d, int h) {
  const uint32_t u = (h ? d >> 16 : d & 0xFFFFu);
  return TYPE == MM_BF16 ? bf16_to_f32(u) : (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}

// Eight codes from one chunk: the integers nearest to x / s (ties to even).
// Adding 1.5 * 2^23 rounds x * inv to an integer q, within one of the wanted
// (|x| <= 127.5 s, inv = 127 / amax).  The remainder x - q s is a multiple of
// s's last place (or of x's, if that is finer) below 2^25 of them, so the fma
// gives it exactly: q is right unless it reaches s / 2, and then (a tie, or a
// neighbour, in hardly any chunk) the comparison decides.
template <int TYPE>
__device__ __forceinline__ void quant_chunk(v4i v, float s, float inv, float up, uint32_t *o) {
  constexpr float kMagic = 12582912.0f;
  float f[8], q[8], far = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    f[j] = row_elem<TYPE>((uint32_t)v[j >> 1], j & 1) * up;
    q[j] = fmaf(f[j], inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(kMagic - q[j], s, f[j])));
  }
  if (__builtin_expect(2.0f * far >= s, 0)) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      float n = q[j] - kMagic;
      const float e = 2.0f * fmaf(-n, s, f[j]);
      const bool odd = (int)n & 1;
      if (e > s || (e == s && odd)) n += 1.0f;
      else if (e < -s || (e == -s && odd)) n -= 1.0f;
      q[j] = __builtin_amdgcn_fmed3f(n, -127.0f, 127.0f) + kMagic;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; h++) {          // the low byte of q's bits is the code
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(q[4 * h + 1]), __float_as_uint(q[4 * h]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(q[4 * h + 3]), __float_as_uint(q[4 * h + 2]), 0x0c0c0400u);
    o[h] = lo | hi << 16;
  }
}

typedef uint16_t v2us __attribute__((ext_vector_type(2)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// Largest magnitude bits of a chunk in either half, folded into m.
__device__ __forceinline__ v2us quant_largest(v2us m, v4i v) {
#pragma unroll
  for (int d = 0; d < 4; d++)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(v2us, (uint32_t)v[d] & 0x7FFF7FFFu));
  return m;
}

// Scale of a row from its largest magnitude's bits, and what its codes need.
struct RowScale {
  float scale, s, inv, up;
  bool zero;
};
template <int TYPE>
__device__ __forceinline__ RowScale row_scale(uint32_t m) {
  RowScale r;
  const bool bad = m >= (TYPE == MM_BF16 ? 0x7F80u : 0x7C00u);
  const float amax = row_elem<TYPE>(m, 0);
  r.scale = bad ? __uint_as_float(0x7FC00000u) : amax / 127.0f;
  r.zero = bad || r.scale == 0.0f;
  // rows too small for 127 / amax to stay in range are worked 2^64 larger (exact)
  r.up = amax < 1e-30f ? 0x1p64f : 1.0f;
  r.s = r.scale * r.up;
  r.inv = r.zero ? 0.0f : 127.0f / (amax * r.up);
  return r;
}

// One block per row, a chunk of eight values a thread (rows past 8192 columns
// take turns, and are read twice): the row's largest magnitude, then its codes.
// One chunk a thread keeps the code short, which is what a few rows cost
// (8 rows of 7168: 3.5 us, 6.4 us with four chunks on 256 threads).  A row
// with an infinity or NaN gets scale NaN and codes 0, so its products are NaN.
template <int TYPE>
__global__ __launch_bounds__(1024) void k_quant_int8(const uint16_t *x, long rows, int cols, int8_t *q, float *scales) {
  __shared__ uint32_t red[16];
  const int n = cols / 8, tid = threadIdx.x, step = blockDim.x;
  for (size_t row = blockIdx.x; row < (size_t)rows; row += gridDim.x) {
    const v4i *src = (const v4i *)(x + row * cols);
    v2u *dst = (v2u *)(q + row * cols);
    v2us mm = {0, 0};
    v4i v = {0, 0, 0, 0};
    for (int i = tid; i < n; i += step) {
      v = src[i];
      mm = quant_largest(mm, v);
    }
    uint32_t m = row16_max(max((uint32_t)mm[0], (uint32_t)mm[1]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (step > 64) {
      __syncthreads();                   // the row before is done with red
      if ((tid & 63) == 0) red[tid >> 6] = m;
      __syncthreads();
      m = row16_max((tid & 15) < (step >> 6) ? red[tid & 15] : 0);
    }
    const RowScale r = row_scale<TYPE>(m);
    if (tid == 0) scales[row] = r.scale;
    for (int i = tid; i < n; i += step) {
      if (n > step) v = src[i];
      uint32_t o[2];
      quant_chunk<TYPE>(v, r.s, r.inv, r.up, o);
      dst[i] = r.zero ? v2u{0, 0} : v2u{o[0], o[1]};
    }
  }
}

// Many rows: W waves per row that they hold in registers, two chunks a lane, and
// several rows a block where W is small.  More chunks a lane leave too few waves
// to load, compute and store at the same time, fewer make the barrier and the
// start of a row count: 4096 rows of 4096 in 12.6 us with two, 13.8 with four,
// 16.2 with eight; of 7168 in 20.0 us (4.4 TB/s) with two, 26.3 with sixteen.  The
// kernel above takes 15.2 and 29.7 us there, and is as fast at 1024 rows.
template <int TYPE, int W>
__global__ __launch_bounds__(W > 4 ? 64 * W : 256) void k_quant_int8_rows(const uint16_t *x, long rows, int cols,
                                                                        int8_t *q, float *scales) {
  constexpr int CH = 2, NR = W > 4 ? 1 : 4 / W;
  __shared__ uint32_t red[2][NR * W];
  const int n = cols / 8, w = threadIdx.x >> 6, at = (w % W) * 64 + (threadIdx.x & 63);
  int turn = 0;
  for (long base = (long)blockIdx.x * NR; base < rows; base += (long)gridDim.x * NR, turn ^= 1) {
    const long row = base + w / W;
    const int mine = row < rows ? n : 0;
    const v4i *src = (const v4i *)(x + row * cols);
    v2u *dst = (v2u *)(q + row * cols);
    v4i v[CH];
#pragma unroll
    for (int i = 0; i < CH; i++) v[i] = at + 64 * W * i < mine ? src[at + 64 * W * i] : v4i{0, 0, 0, 0};
    v2us mm = {0, 0};
#pragma unroll
    for (int i = 0; i < CH; i++) mm = quant_largest(mm, v[i]);
    uint32_t m = row16_max(max((uint32_t)mm[0], (uint32_t)mm[1]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if constexpr (W > 1) {               // two turns' slots: one barrier a turn
      if ((threadIdx.x & 63) == 0) red[turn][w] = m;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < W; k++) m = max(m, red[turn][w / W * W + k]);
    }
    const RowScale r = row_scale<TYPE>(m);
    if (at == 0 && mine) scales[row] = r.scale;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      if (at + 64 * W * i >= mine) break;
      uint32_t o[2];
      quant_chunk<TYPE>(v[i], r.s, r.inv, r.up, o);
      dst[at + 64 * W * i] = r.zero ? v2u{0, 0} : v2u{o[0], o[1]};
    }
  }
}

constexpr long kQuantBlocks = 1 << 18;   // most blocks of a launch: longer batches take further turns

template <int TYPE, int W>
static void launch_quant_rows(const uint16_t *x, long rows, int cols, int8_t *q, float *scales, hipStream_t s) {
  constexpr int NR = W > 4 ? 1 : 4 / W;
  hipLaunchKernelGGL((k_quant_int8_rows<TYPE, W>), dim3((unsigned)std::min((rows + NR - 1) / NR, kQuantBlocks)),
                     dim3(64 * NR * W), 0, s, x, rows, cols, q, scales);
}

template <int TYPE>
static hipError_t launch_quant(const uint16_t *x, long rows, int cols, int8_t *q, float *scales, hipStream_t s) {
  const int n = cols / 8;
  if (rows >= 2048 && n <= 2048) {
    if (n <= 128) launch_quant_rows<TYPE, 1>(x, rows, cols, q, scales, s);
    else if (n <= 256) launch_quant_rows<TYPE, 2>(x, rows, cols, q, scales, s);
    else if (n <= 512) launch_quant_rows<TYPE, 4>(x, rows, cols, q, scales, s);
    else if (n <= 1024) launch_quant_rows<TYPE, 8>(x, rows, cols, q, scales, s);
    else launch_quant_rows<TYPE, 16>(x, rows, cols, q, scales, s);
  } else {
    const dim3 t(cols >= 8192 ? 1024 : (n + 63) / 64 * 64);
    hipLaunchKernelGGL(k_quant_int8<TYPE>, dim3((unsigned)std::min(rows, kQuantBlocks)), t, 0, s, x, rows, cols, q, scales);
  }
  return hipGetLastError();
}

hipError_t launch_quant_int8(int type, const void *x, long rows, int cols, int8_t *q, float *scales, hipStream_t s) {
  return type == MM_BF16 ? launch_quant<MM_BF16>((const uint16_t *)x, rows, cols, q, scales, s)
                         : launch_quant<MM_FP16>((const uint16_t *)x, rows, cols, q, scales, s);
}

// ------------------------------------------------------------ grouping

constexpr int kGroupMaxE = 1024;   // one thread of a block per expert
constexpr int kGroupWaves = kGroupThreads / 64;

__device__ __forceinline__ int group_id(const GroupArgs &a, int r) {
  const int e = r < a.R ? a.ids[r] : -1;
  return e >= 0 && e < a.E ? e : -1;
}

// Outputs of route r, at sorted row pos when its id e is an expert's.  The
// rows behind the last group are as many as the routes without an expert.
__device__ __forceinline__ void group_place(const GroupArgs &a, int r, int e, int pos, int rows) {
  if (r >= a.R) return;
  a.inverse[r] = e < 0 ? -1 : pos;
  if (e >= 0) {
    a.order[pos] = r;
    a.token[pos] = r / a.topk;
  }
  if (r >= rows) a.order[r] = a.token[r] = -1;
}

// Few routes (R and E at most the block's threads): every thread compares its expert and its route with all ids in
// LDS, so offsets and sorted rows come without counting or scanning (one
// barrier instead of five: 8 tokens of top-6 over 384 experts in 3.9 us
// against 7.1 us by a counting kernel).
__global__ __launch_bounds__(kGroupThreads) void k_group_few(GroupArgs a) {
  __shared__ __align__(16) int ids[kGroupFew];
  const int tid = threadIdx.x;
  for (int i = tid; i < kGroupFew; i += blockDim.x) {
    const int e = group_id(a, i);
    ids[i] = e < 0 ? INT32_MAX : e;     // sorts behind every expert
  }
  __syncthreads();
  const int mine = tid < a.R ? ids[tid] : INT32_MAX;
  int below = 0, pos = 0, rows = 0;     // routes of experts before tid; routes before this one; routes with an expert
  const int n4 = (a.R + 3) >> 2;
  for (int i = 0; i < n4; i++) {
    const v4i v = ((const v4i *)ids)[i];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      below += v[j] < tid;
      rows += v[j] < a.E;
      pos += v[j] < mine || (v[j] == mine && 4 * i + j < tid);
    }
  }
  if (tid < a.E) a.first[tid] = below;
  if (tid == 0) a.first[a.E] = rows;
  group_place(a, tid, mine == INT32_MAX ? -1 : mine, pos, rows);
}

// Counting sort.  A wave's routes of one expert are found together by ballots
// over the bits of the id; a route's rank is its number among them, plus the
// block's routes of the expert in earlier waves and rounds.
struct GroupLds {
  uint16_t whist[kGroupWaves][kGroupMaxE];
  int cnt[kGroupMaxE], off[kGroupMaxE + 1], wsum[kGroupWaves];
};

// One round of kGroupThreads routes: rank of this thread's route (id e, -1:
// none) among the block's routes of its expert; cnt[] moves on by the round.
__device__ __forceinline__ int group_round(GroupLds &L, int E, int bits, int e) {
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  for (int i = tid; i < E; i += kGroupThreads)
#pragma unroll
    for (int v = 0; v < kGroupWaves; v++) L.whist[v][i] = 0;
  __syncthreads();
  unsigned long long same = __ballot(e >= 0);
  for (int b = 0; b < bits; b++) {
    const unsigned long long m = __ballot((e >> b) & 1);
    same &= ((e >> b) & 1) ? m : ~m;
  }
  int rank = __popcll(same & ((1ull << lane) - 1ull));
  if (e >= 0 && rank == 0) L.whist[w][e] = (uint16_t)__popcll(same);
  __syncthreads();
  if (tid < E) {
    int run = L.cnt[tid];
#pragma unroll
    for (int v = 0; v < kGroupWaves; v++) {
      const int c = L.whist[v][tid];
      L.whist[v][tid] = (uint16_t)(run - L.cnt[tid]);
      run += c;
    }
    L.off[tid] = L.cnt[tid];           // the block's count before this round
    L.cnt[tid] = run;
  }
  __syncthreads();
  if (e >= 0) rank += L.whist[w][e] + L.off[e];
  __syncthreads();
  return rank;
}

// off[0 .. E] from cnt[0 .. E), one thread per expert.
__device__ __forceinline__ void group_offsets(GroupLds &L, int E) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int c = tid < E ? L.cnt[tid] : 0;
  int s = c;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(s, d);
    if (lane >= d) s += v;
  }
  if (lane == 63) L.wsum[tid >> 6] = s;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int v = 0; v < kGroupWaves; v++) before += v < (tid >> 6) ? L.wsum[v] : 0;
  if (tid < E) L.off[tid] = before + s - c;
  if (tid == E - 1) L.off[E] = before + s;
  __syncthreads();
}

// ROUNDS > 0: one block sorts all of ROUNDS * kGroupThreads routes at most.
// ROUNDS == 0: the block counts its share (a.rounds rounds), counts and ranks to scratch.
template <int ROUNDS>
__global__ __launch_bounds__(kGroupThreads) void k_group(GroupArgs a) {
  __shared__ GroupLds L;
  const int tid = threadIdx.x;
  const int bits = 32 - __clz(a.E);
  if (tid < a.E) L.cnt[tid] = 0;
  if constexpr (ROUNDS > 0) {
    int e[ROUNDS], rank[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; i++) e[i] = group_id(a, i * kGroupThreads + tid);
#pragma unroll
    for (int i = 0; i < ROUNDS; i++) rank[i] = group_round(L, a.E, bits, e[i]);
    group_offsets(L, a.E);
    for (int i = tid; i <= a.E; i += kGroupThreads) a.first[i] = L.off[i];
#pragma unroll
    for (int i = 0; i < ROUNDS; i++)
      group_place(a, i * kGroupThreads + tid, e[i], e[i] < 0 ? 0 : L.off[e[i]] + rank[i], L.off[a.E]);
  } else {
    const int r0 = blockIdx.x * a.rounds * kGroupThreads + tid;
    int e = group_id(a, r0);
    for (int i = 0; i < a.rounds; i++) {
      const int r = r0 + i * kGroupThreads;
      const int next = i + 1 < a.rounds ? group_id(a, r + kGroupThreads) : -1;
      const int rank = group_round(L, a.E, bits, e);
      if (r < a.R) a.rank[r] = rank;
      e = next;
    }
    if (tid < a.E) a.hist[(size_t)blockIdx.x * a.E + tid] = L.cnt[tid];
  }
}

// Placement of one block's share.  Each block sums the blocks' counts itself,
// all of them and those before its own (at most kGroupMaxBlocks * E values,
// from L2), which saves the launch of a scan.
__global__ __launch_bounds__(kGroupThreads) void k_group_place(GroupArgs a) {
  __shared__ GroupLds L;
  __shared__ int before[kGroupMaxE];
  const int tid = threadIdx.x;
  if (tid < a.E) L.cnt[tid] = before[tid] = 0;
  __syncthreads();
  // threads split over E columns and, when E is small, shares of the blocks
  const int parts = max(1, kGroupThreads / a.E), part = tid / a.E, e0 = tid - part * a.E;
  if (part < parts) {
    int all = 0, mine = 0;
#pragma unroll 8
    for (int c = part; c < a.blocks; c += parts) {
      const int v = a.hist[(size_t)c * a.E + e0];
      all += v;
      mine += c < (int)blockIdx.x ? v : 0;
    }
    atomicAdd(&L.cnt[e0], all);        // integers: the order does not matter
    atomicAdd(&before[e0], mine);
  }
  __syncthreads();
  group_offsets(L, a.E);
  if (blockIdx.x == 0)
    for (int i = tid; i <= a.E; i += kGroupThreads) a.first[i] = L.off[i];
  const int r0 = blockIdx.x * a.rounds * kGroupThreads + tid;
  for (int i = 0; i < a.rounds; i++) {
    const int r = r0 + i * kGroupThreads, e = group_id(a, r);
    group_place(a, r, e, e < 0 ? 0 : L.off[e] + before[e] + a.rank[r], L.off[a.E]);
  }
}

hipError_t launch_group(const GroupArgs &a, hipStream_t s) {
  const dim3 t(kGroupThreads);
  if (a.R <= kGroupFew) {
    const int n = a.E > a.R ? a.E : a.R;
    hipLaunchKernelGGL(k_group_few, dim3(1), dim3((n + 63) / 64 * 64), 0, s, a);
  } else if (a.R <= kGroupThreads) {
    hipLaunchKernelGGL(k_group<1>, dim3(1), t, 0, s, a);
  } else if (a.R <= 4 * kGroupThreads) {
    hipLaunchKernelGGL(k_group<4>, dim3(1), t, 0, s, a);
  } else {
    hipLaunchKernelGGL(k_group<0>, dim3(a.blocks), t, 0, s, a);
    hipLaunchKernelGGL(k_group_place, dim3(a.blocks), t, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
