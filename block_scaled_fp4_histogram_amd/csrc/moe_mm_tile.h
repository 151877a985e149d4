// Kernel templates of the ragged products for gfx950: tiles and streamed weights,
// shared by the plain products (moe_mm.hip), the gated block (moe_glu.hip) and the
// 8-bit floating-point products (moe_fp8.hip).
#pragma once

#include "moe_device.h"
#include "moe_glu.h"
#include "moe_mm.h"

namespace moe {

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

// 8-bit floating point (E4M3): the operands hold 128 of the reduction, a block of one
// scale, so a product of them from zero is that block's sum.
//
// MM_F8X: the codes as fp16 values, which is exact, in fp16 instructions, which sum in
// fp32.
// MM_F8, where the caller asks for it: one instruction.  Inside it the products of eight
// consecutive values (a register pair of either operand) meet with what lies 13 bits and
// more below the largest of them cut off, and the eights' sums meet in fp32 (measured on
// all their positions; the instruction for 32 values of the reduction does the same).
// That is 2^-10 of a block's magnitudes at worst, all of a sum whose large products
// cancel, and about 5e-5 of a random sum; the rate is twice that of any instruction that
// keeps fp32.  It applies the powers of two of the block's scales itself.
template <>
struct MmElem<MM_F8> {
  typedef uint8_t t;
  typedef v4f acc;
};
template <>
struct MmElem<MM_F8X> : MmElem<MM_F8> {};
__device__ __forceinline__ v8i join8(v4i lo, v4i hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
// Eight codes as fp16.
__device__ __forceinline__ v8h codes_f16(int lo, int hi) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)lo, 1.0f, true);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)hi, 1.0f, true);
  return v8h{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A block's scale as the E8M0 code of a power of two, which is its exponent's bits, and
// a factor of magnitude in [1, 2): less for subnormal scales, and 0 with the least power
// of two for 0, so that no sum is infinite before it meets the 0.  (Infinite and NaN
// scales have E8M0's NaN.)  The sum meets the powers of two and the factors' product
// apart, so the product of two scales never leaves fp32's range before the result does.
struct MmScale8 {
  float m;
  int code;
};
__device__ __forceinline__ MmScale8 mm_scale8(float s) {
  const int code = (int)((__float_as_uint(s) >> 23) & 0xFFu);
  return MmScale8{__builtin_ldexpf(s, 127 - code), code};
}
constexpr int kF8Block = 128;            // values of a scale, along either side
// The same as two factors, first * second, that a block's sum (2^-18 to 2^25) meets in turn:
// the first within 2^100 of 1 (but for subnormal scales' fractions), so that the sum times it
// loses nothing that the result has, and the second 1 unless the scales' product is further off.
__device__ __forceinline__ void mm_factors8(MmScale8 w, MmScale8 x, float &first, float &second) {
  const int e = w.code + x.code - 254, near = min(max(e, -100), 100);
  first = __builtin_ldexpf(w.m * x.m, near);
  second = __builtin_ldexpf(1.0f, min(max(e - near, -126), 127));
}

// acc + a block's sum times its scales.
__device__ __forceinline__ v4f f8_block(v4f acc, v8i p, v8i q, MmScale8 w, MmScale8 x) {
  float first, second;
  mm_factors8(w, x, first, second);
  v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 4; k++) d = mfma_f16(codes_f16(p[2 * k], p[2 * k + 1]), codes_f16(q[2 * k], q[2 * k + 1]), d);
#pragma unroll
  for (int k = 0; k < 4; k++) acc[k] = fmaf(d[k] * first, second, acc[k]);
  return acc;
}

// Two results in one register, each rounded to nearest even.
template <int OUT>
__device__ __forceinline__ uint32_t mm_pack(float lo, float hi) {
  if (OUT == MM_BF16) return pack_bf16x2(lo, hi);
  return __builtin_bit_cast(uint32_t, v2h{(_Float16)lo, (_Float16)hi});
}

typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// NT: past the caches' keeping.
template <bool NT, typename V>
__device__ __forceinline__ void mm_store(V *o, V v) {
  if (NT) __builtin_nontemporal_store(v, o);
  else *o = v;
}

template <bool NT = false>
__device__ __forceinline__ void mm_store_f32(const MmArgs &a, long at, v4f r) {
  v4f *o = (v4f *)((float *)a.out + at);
  if (a.accumulate) r += *o;
  mm_store<NT>(o, r);
}

// Four or eight consecutive results (8- or 16-byte aligned in the output's type).
template <int OUT>
__device__ __forceinline__ void mm_store4(const MmArgs &a, long at, const float *v) {
  if (OUT == MM_FP32) mm_store_f32(a, at, v4f{v[0], v[1], v[2], v[3]});
  else *(v2u *)((uint16_t *)a.out + at) = v2u{mm_pack<OUT>(v[0], v[1]), mm_pack<OUT>(v[2], v[3])};
}

template <int OUT>
__device__ __forceinline__ void mm_store8(const MmArgs &a, long at, const float *v) {
  if (OUT == MM_FP32) {
    mm_store4<OUT>(a, at, v);
    mm_store4<OUT>(a, at + 4, v + 4);
  } else {
    typedef uint32_t v4u __attribute__((ext_vector_type(4)));
    const v4u r = v4u{mm_pack<OUT>(v[0], v[1]), mm_pack<OUT>(v[2], v[3]), mm_pack<OUT>(v[4], v[5]),
                      mm_pack<OUT>(v[6], v[7])};
    *(v4u *)((uint16_t *)a.out + at) = r;
  }
}

// An integer sum by the scales of its row and channel.  The scales' fractions meet in
// [1/4, 1) and their exponents are applied last, so neither the scales' product nor a
// scale's with the sum leaves fp32's range before the result does (1e-22 * 1e-22 * 1e9;
// 2.4e36 * 200 * 0), and where nothing leaves it the result is sum * (x * w) bit for bit.
struct MmScale {
  float m;
  int e;
};
__device__ __forceinline__ MmScale mm_scale(float s) {
  return MmScale{__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)};
}
__device__ __forceinline__ float mm_scaled(int sum, MmScale x, MmScale w) {
  return __builtin_ldexpf((float)sum * (x.m * w.m), x.e + w.e);
}

typedef __attribute__((address_space(4))) const float MmConstF;   // read by scalar loads

// f(integral constant of the output type): the branch on it stands outside the stores.
template <int V>
struct MmConst {
  static constexpr int value = V;
};
constexpr int MM_PART = 5;   // 32-bit sums of one part of the reduction, as they are
template <int TYPE, typename F>
__device__ __forceinline__ void mm_by_output(int out_type, F f) {
  if (out_type == MM_PART) f(MmConst<MM_PART>{});
  else if (TYPE != MM_F8 && out_type == MM_FP32) f(MmConst<MM_FP32>{});   // (MM_F8 has 16-bit results)
  else if (out_type == MM_BF16) f(MmConst<MM_BF16>{});
  else f(MmConst<MM_FP16>{});
}

// ------------------------------------------------------------ tile kernels

typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr uint32_t kOutside = 0x80000000u;   // lane offset past every resource: loads zeros

// A gathered row that names no row of x, and the part of a row past its end,
// are read from here.
static __device__ const uint32_t g_mm_zeros[4] = {0, 0, 0, 0};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ Rsrc mm_rsrc(const uint8_t *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)bytes, 0x00020000);
}

// A barrier that LDS accesses are not moved across; the waits are the caller's.
__device__ __forceinline__ void mm_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Row range of group e.
__device__ __forceinline__ void mm_group(const MmArgs &a, int e, int &lo, int &hi) {
  if (!a.first) {
    lo = 0;
    hi = a.R;
  } else {
    lo = min(max(a.first[e], 0), a.R);
    hi = min(max(a.first[e + 1], lo), a.R);
  }
}

// Inclusive scan over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

struct MmTile {
  int e, row0, rows, pt;   // group, first row, rows of the tile; column tile
};

// The products by their operands: forward ones take rows of x and of w as they lie,
// row gradients (of dy and w) and weight gradients read theirs transposed.
constexpr bool mm_forward(int op) { return op == MM_FORWARD || op == MM_GLU; }
constexpr bool mm_dx(int op) { return op == MM_DX || op == MM_GLU_DX; }
// The gated block's products and 8-bit floating point; of these the shapes whose last round
// may be in parts (of two blocks a CU: the plan takes no other).
constexpr bool mm_built(int op, int type) { return op == MM_GLU || op == MM_GLU_DX || type == MM_F8 || type == MM_F8X; }
constexpr bool mm_has_tail(int op, int type, int bq, int bp) { return mm_built(op, type) && bq * bp == 256 * 128; }
// Columns of the output, and of a tile of BP rows of w: the gated block's come from two.
__host__ __device__ __forceinline__ constexpr int mm_outs(int op, int N, int K) { return mm_forward(op) ? N : K; }
constexpr int mm_tile_cols(int op, int bp) { return op == MM_GLU ? bp / 2 : bp; }

// The output tile of this block, from the offsets on the GPU.  Row tiles of BQ
// rows are numbered over the groups in order; a lane counts the tiles of
// E / 64 consecutive groups, one scan gives the total, a second over the found
// lane's groups the tile's own.  Blocks go to the eight XCDs in turn, so XCD i
// takes the i-th eighth of the tiles that exist (not of the launch's upper
// bound, whose surplus blocks would all land on the last XCD), and inside it
// kMmGroup row tiles share each column tile of the weights before the next one
// is read (16384 x 4096 x 4096 with 1, 4, 8 and 16: 485, 428, 431, 462 us; eight
// groups' row gradient of that size: 488, 505, 497, 530).  Every wave does the same work: no barrier.
constexpr int kMmGroup = 8;

// pick(number of tiles): this block's tile, or -1.
template <int BQ, typename Pick>
__device__ __forceinline__ bool mm_tile_by(const MmArgs &a, int ptiles, MmTile &t, Pick pick) {
  const int lane = threadIdx.x & 63;
  if (!a.first) {                        // one group: the same order without the scans
    const int total = (a.R + BQ - 1) / BQ, id = pick(total * ptiles);
    if (id < 0) return false;
    const int grp = id / (kMmGroup * ptiles), rem = id - grp * kMmGroup * ptiles;
    const int gcur = min(kMmGroup, total - grp * kMmGroup);
    t.e = 0;
    t.pt = rem / gcur;
    t.row0 = (grp * kMmGroup + rem % gcur) * BQ;
    t.rows = min(BQ, a.R - t.row0);
    return true;
  }
  const int per = (a.E + 63) >> 6;
  int cnt = 0, lo = 0, hi = 0;
  if (per == 1) {
    if (lane < a.E) mm_group(a, lane, lo, hi);
    cnt = (hi - lo + BQ - 1) / BQ;
  } else {                               // eight groups' offsets at once: one wait for them all
    for (int i = 0; i < per; i += 8) {
      int v[9];
#pragma unroll
      for (int k = 0; k < 9; k++) v[k] = a.first[min(lane * per + i + k, a.E)];
#pragma unroll
      for (int k = 0; k < 8; k++) {
        if (i + k >= per) break;
        lo = min(max(v[k], 0), a.R);
        hi = min(max(v[k + 1], lo), a.R);
        cnt += (hi - lo + BQ - 1) / BQ;
      }
    }
  }
  const int sum = wave_scan(cnt);
  const int total = uniform(__shfl(sum, 63));
  // (a total below zero: offsets that fall, whose groups overlap past 2^31 tiles)
  const int id = total <= 0 ? -1 : pick(total * ptiles);
  if (id < 0) return false;
  const int grp = id / (kMmGroup * ptiles), rem = id - grp * kMmGroup * ptiles;
  const int gcur = min(kMmGroup, total - grp * kMmGroup);
  t.pt = rem / gcur;
  const int rt = grp * kMmGroup + rem % gcur;
  const int src = __ffsll(__ballot(sum > rt)) - 1;
  const int before = __shfl(sum - cnt, src);
  int at = 0, k = rt - before;           // the group's number in the lane's, its tile
  if (per == 1) {
    at = src;
  } else {
    const int e = src * per + lane;
    lo = hi = 0;
    if (lane < per && e < a.E) mm_group(a, e, lo, hi);
    const int c = (hi - lo + BQ - 1) / BQ, s2 = wave_scan(c);
    at = __ffsll(__ballot(before + s2 > rt)) - 1;
    k -= __shfl(s2 - c, at);
  }
  t.e = uniform(per == 1 ? src : src * per + at);
  t.row0 = uniform(__shfl(lo, at) + k * BQ);
  t.rows = min(BQ, uniform(__shfl(hi, at)) - t.row0);
  return t.rows > 0;
}

// Tile of block b of n that each XCD takes an eighth of, or -1.
__device__ __forceinline__ int mm_eighths(int b, int n) {
  const int chunk = (n + 7) >> 3, id = (b & 7) * chunk + (b >> 3);
  return (b >> 3) >= chunk || id >= n ? -1 : id;
}
template <int BQ>
__device__ __forceinline__ bool mm_find_tile(const MmArgs &a, int ptiles, MmTile &t) {
  return mm_tile_by<BQ>(a, ptiles, t, [](int nt) { return mm_eighths((int)blockIdx.x, nt); });
}

// The last round of a launch of more than one.  Where its tiles would fill half of the
// chip's slots or less, each is taken by several blocks, which split its reduction and
// leave their sums in scratch for k_tail_join to add in order.  (Groups of unequal size
// make any number of tiles: 32 experts' 16384 rows are 512 tiles of 256 x 128 if all
// have the same number, one round in 228 us, and 640 with loads of rank^-0.5, 381 us.)
// full: tiles before them, taken whole; rem: tiles of the last round; parts of each (1: whole).
constexpr int kTailParts = 8, kTailSteps = 8;      // most parts of a tile, fewest steps of a part
struct MmTail {
  int full, rem, parts;
};
__host__ __device__ __forceinline__ MmTail mm_tail(int nt, int slots, int steps) {
  const int full = nt / slots * slots, rem = nt - full;
  int parts = rem ? slots / rem : 1;
  parts = parts < kTailParts ? parts : kTailParts;
  parts = parts < steps / kTailSteps ? parts : steps / kTailSteps;
  if (parts < 2) return MmTail{nt, 0, 1};
  return MmTail{full, rem, parts};
}

// Row of x behind product row r, or -1.
__device__ __forceinline__ long mm_x_row(const MmArgs &a, int r) {
  if (!a.rows) return r;
  const int x = a.rows[r];
  return x >= 0 && x < a.x_rows ? (long)x : -1l;
}

// LDS images of an operand tile, 128 bytes of the reduction (one step) by B
// outer indices.  Reduction-contiguous operands: B rows of eight 16-byte
// chunks, chunk c of row r at slot c ^ swz(r); transposed ones: 64 rows of B
// 16-bit columns, chunk c of row z at c ^ 2 swz(z).  Either way the 16 (or,
// transposed, 32) lanes that read together touch every bank once.
//   Contiguous rows are read 16 consecutive ones a fragment: bits 1 to 3 of r.
//   Transposed rows are read 8 g .. 8 g + 3 by lane group g, and 4 further on
//   next: bits 0, 1 and 3 of z.
__device__ __forceinline__ int swz_r(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int swz_t(int z) { return (z & 3) | ((z >> 1) & 4); }

// The MFMA's rows are the output's contiguous dimension (P: weights, or x for
// the weight gradient), its columns the output's rows (Q), so a lane's four
// results are contiguous.
template <int OP, int TYPE, int BQ, int BP, int WQ, int WP, bool GATHER, int MINW>
__global__ __launch_bounds__(64 * WQ * WP, MINW) void k_mm_tile(MmArgs a) {
  typedef MmElem<TYPE> M;
  constexpr int ES = sizeof(typename M::t), NW = WQ * WP;
  constexpr bool FWD = mm_forward(OP), DX = mm_dx(OP), GLU = OP == MM_GLU, F8 = TYPE == MM_F8 || TYPE == MM_F8X;
  constexpr bool TQ_T = OP == MM_DW, TP_T = !FWD;               // transposed operands
  constexpr int TQ = BQ / WQ, TP = BP / WP, NQ = TQ / 16, NP = TP / 16;
  constexpr int CQ = BQ / 8 / NW, CP = BP / 8 / NW;             // loads of 1 KB a wave and step
  constexpr int kStage = (BQ + BP) * 128;
  static_assert(TP % 64 == 0 && TQ % 16 == 0 && CQ >= 1 && CP >= 1, "tile shape");
  static_assert(!TQ_T || (BQ % 128 == 0 && TQ % 64 == 0), "transposed Q");
  static_assert(!TP_T || BP % 128 == 0, "transposed P");
  constexpr int kOutStage = 16 * (64 * 4 + 16);                 // of one wave, for its outputs
  static_assert(NW * kOutStage <= kStage, "outputs through LDS");
  __shared__ __align__(1024) uint8_t lds[kStage];
  __shared__ __align__(16) float xsl[F8 ? 2 * BQ * 4 : 4];      // scales of x's rows: twice four blocks of K

  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  constexpr int BC = mm_tile_cols(OP, BP);
  const int pn = mm_outs(OP, a.N, a.K);                         // output columns
  const int ptiles = (pn + BC - 1) / BC;
  MmTile t;
  int q0 = 0, qn, zn;                                           // output rows of the tile, reduction
  // of the products built on these, in their largest shapes: a tile of the last round in parts (mm_tail)
  constexpr bool TAIL = mm_has_tail(OP, TYPE, BQ, BP);
  int part = 0, parts = 1, tail_at = 0;                         // this block's part, and its tile's number among them
  if (OP == MM_DW) {
    // each group's tiles spread over the XCDs, so that a large group does not load one of them
    const int tiles = ((a.N + BQ - 1) / BQ) * ptiles, per8 = (tiles + 7) >> 3;
    const int b = (int)blockIdx.x >> 3, id = ((int)blockIdx.x & 7) * per8 + b % per8;
    t.e = b / per8;
    if (id >= tiles) return;
    t.pt = id % ptiles;
    q0 = (id / ptiles) * BQ;
    int lo, hi;
    mm_group(a, t.e, lo, hi);
    t.row0 = uniform(lo);
    t.rows = uniform(hi) - t.row0;
    if (a.accumulate && t.rows == 0) return;   // nothing to add: what dw holds stays as it is
    qn = min(BQ, a.N - q0);
    zn = t.rows;
  } else {
    if (TAIL && a.tail) {
      const int reduction = FWD ? a.K : a.N, all = (reduction + 128 / ES - 1) / (128 / ES);
      const bool any = mm_tile_by<BQ>(a, ptiles, t, [&](int nt) {
        const MmTail m = mm_tail(nt, 256 * MINW, all);
        const int b = (int)blockIdx.x;
        if (m.rem == 0 || b < m.full) return mm_eighths(b, m.full);
        const int u = mm_eighths(b - m.full, m.rem * m.parts);
        if (u < 0) return -1;
        part = u / m.rem, parts = m.parts, tail_at = u % m.rem;
        return m.full + tail_at;
      });
      if (!any) return;
      part = uniform(part), parts = uniform(parts), tail_at = uniform(tail_at);
    } else if (!mm_find_tile<BQ>(a, ptiles, t)) {
      return;
    }
    if constexpr (F8) {                  // (in scalar registers from here on, or the loads loop over their lanes' resources)
      t.row0 = uniform(t.row0), t.rows = uniform(t.rows);
      t.e = uniform(t.e), t.pt = uniform(t.pt);
    }
    qn = t.rows;
    zn = FWD ? a.K : a.N;
  }
  const int p0 = t.pt * BC;
  constexpr int ZS = (TQ_T || TP_T) ? 64 : 128 / ES;            // reduction elements a step
  // with a split reduction, this block's share of the steps
  const int all = (zn + ZS - 1) / ZS, cut = TAIL && parts > 1 ? parts : a.splits, share = cut > 1 ? (all + cut - 1) / cut : all;
  const int begin = (TAIL && parts > 1 ? part : (int)blockIdx.y) * share, steps = min(all, begin + share);

  // ---- loads of one step
  const uint8_t *x = (const uint8_t *)a.x, *dy = (const uint8_t *)a.dy;
  const uint8_t *wt = (const uint8_t *)a.w + (size_t)t.e * (GLU ? 2 * a.N : a.N) * a.K * ES;
  const uint32_t ldx = (uint32_t)a.K * ES, ldy = (uint32_t)a.N * ES;

  // A wave's loads of an operand are the same lanes of rows a fixed step apart,
  // so one offset a lane does for all of them.  Contiguous operands: load i holds
  // rows (i NW + w) 8 + lane / 8; transposed ones, LR lanes a row: rows
  // (i NW + w) 64 / LR + lane / LR.
  constexpr int LRQ = BQ / 8, LRP = BP / 8;
  constexpr int DQ = TQ_T ? NW * 64 / LRQ : NW * 8, DP = TP_T ? NW * 64 / LRP : NW * 8;   // rows between loads
  // The swizzle repeats over a wave's loads, but for one bit of it that flips with
  // every load where the rows between them reach only that bit: these bytes.
  static_assert(TQ_T ? DQ % 8 == 0 : DQ % 16 == 0, "loads of Q");
  static_assert(TP_T ? DP % 8 == 0 : DP % 16 == 0, "loads of P");
  constexpr uint32_t FQ = TQ_T && DQ % 16 ? 128 : 0, FP = TP_T && DP % 16 ? 128 : 0;
  const int rq0 = TQ_T ? w * (64 / LRQ) + lane / LRQ : w * 8 + (lane >> 3);
  const int rp0 = TP_T ? w * (64 / LRP) + lane / LRP : w * 8 + (lane >> 3);
  // contiguous: the chunk's byte in the step; transposed: its byte in the row
  const uint32_t cq = TQ_T ? q0 * 2 + (((lane % LRQ) ^ (2 * swz_t(rq0))) * 16) : ((lane & 7) ^ swz_r(rq0)) * 16;
  const uint32_t cp = TP_T ? p0 * 2 + (((lane % LRP) ^ (2 * swz_t(rp0))) * 16) : ((lane & 7) ^ swz_r(rp0)) * 16;
  const uint32_t ldq = FWD ? ldx : ldy;
  const uint32_t vq = (uint32_t)rq0 * ldq + cq, vp = (uint32_t)rp0 * ldx + cp;
  const Rsrc rq = FWD  ? mm_rsrc(x + (GATHER ? 0 : (size_t)t.row0 * ldx), (uint32_t)qn * ldx)
                  : DX ? mm_rsrc(dy + (size_t)t.row0 * ldy, (uint32_t)qn * ldy)
                       : mm_rsrc(dy, 0);
  // The gated block's tile holds the gate's rows of w and the up branch's in turn, TP / 2
  // of each, so that a wave has both sums of its columns.
  constexpr int HP = TP / 2;
  static_assert(!GLU || (DP <= HP && HP % DP == 0), "branches of P");
  const Rsrc rp = FWD ? mm_rsrc(wt + (size_t)(p0 + (GLU ? a.glu.gate0 : 0)) * ldx, (uint32_t)min(BC, pn - p0) * ldx) : mm_rsrc(wt, 0);
  // Gathered rows within 2 GiB are loaded through one resource over x, as rows in order are.
  constexpr bool NEAR = GATHER && mm_built(OP, TYPE);
  bool near = false;
  if constexpr (NEAR) near = a.x_rows * (long)ldx < 0x7FFFFFFFl;
  const Rsrc rx = mm_rsrc(x, (uint32_t)(near ? a.x_rows * (long)ldx : 0));
  const Rsrc rup = GLU ? mm_rsrc(wt + (size_t)(p0 + a.glu.up0) * ldx, (uint32_t)min(BC, pn - p0) * ldx) : rp;
  // forward gather: each load's row of x
  constexpr bool GF = GATHER && FWD, GW = GATHER && OP == MM_DW;
  int grow[GF ? CQ : 1];
  if constexpr (GF) {
#pragma unroll
    for (int i = 0; i < CQ; i++) {
      const int r = rq0 + i * DQ;
      grow[i] = r < qn ? (int)mm_x_row(a, t.row0 + r) : -1;
      if constexpr (NEAR) if (near) grow[i] = grow[i] < 0 ? (int)kOutside : (int)((uint32_t)grow[i] * ldx + cq);
    }
  }
  // weight gradient gather: rows of x behind this lane's rows of step s, read one
  // step before they are loaded
  int gidx[GW ? CP : 1];
  auto gather_rows = [&](int s) {
    if constexpr (GW) {
#pragma unroll
      for (int i = 0; i < CP; i++) {
        const int z = s * ZS + rp0 + i * DP;
        gidx[i] = z < zn ? a.rows[t.row0 + z] : -1;
      }
    }
  };
  auto load = [&](int s) {
    uint8_t *lq = lds + w * 1024, *lp = lq + BQ * 128;
    const int left = zn * ES - s * 128;             // contiguous operands: bytes from this step on
    // reduction rows left for transposed operands: rows past them load zeros
    const uint32_t zleft = (uint32_t)min(ZS, zn - s * ZS);
    const Rsrc sq = TQ_T ? mm_rsrc(dy + (size_t)(t.row0 + s * ZS) * ldy, zleft * ldy) : rq;
    const Rsrc sp = DX            ? mm_rsrc(wt + (size_t)(s * ZS) * ldx, zleft * ldx)
                    : OP == MM_DW ? mm_rsrc(x + (size_t)(t.row0 + s * ZS) * ldx, zleft * ldx)
                                  : rp;
#pragma unroll
    for (int i = 0; i < CQ; i++) {
      lds_void *dst = (lds_void *)(lq + i * NW * 1024);
      if constexpr (NEAR) {
        if (near) {
          const Rsrc sx = TQ_T ? sq : rx;   // (a copy, as of the others: the host's pass takes no captured one)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(sx, dst, 16, (int)(NEAR && (int)cq < left ? (uint32_t)grow[GF ? i : 0] : kOutside),
                                                   TQ_T ? 0 : s * 128, 0, 0);
          continue;
        }
      }
      if constexpr (GF) {
        const bool ok = grow[i] >= 0 && (int)cq < left;
        const uint8_t *g = ok ? x + ((size_t)(uint32_t)grow[i] * ldx + (cq + s * 128)) : (const uint8_t *)g_mm_zeros;
        __builtin_amdgcn_global_load_lds(g, dst, 16, 0, 0);
      } else {
        const uint32_t v = vq - cq + (cq ^ (i & 1 ? FQ : 0)) + (uint32_t)(i * DQ) * ldq;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sq, dst, 16, (int)(TQ_T || (int)cq < left ? v : kOutside),
                                                 TQ_T ? 0 : s * 128, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < CP; i++) {
      lds_void *dst = (lds_void *)(lp + i * NW * 1024);
      if constexpr (GW) {
        const uint32_t c = cp ^ (i & 1 ? FP : 0);   // columns past the row's end are not stored
        const bool ok = c < ldx && gidx[i] >= 0 && gidx[i] < a.x_rows;
        const uint8_t *g = ok ? x + ((size_t)(uint32_t)gidx[i] * ldx + c) : (const uint8_t *)g_mm_zeros;
        __builtin_amdgcn_global_load_lds(g, dst, 16, 0, 0);
      } else {
        const uint32_t c = cp ^ (i & 1 ? FP : 0);
        // (gated: the branch of the load's rows, and their columns in it)
        const bool up = GLU && (i * DP / HP & 1);
        const int r0 = GLU ? i * DP / TP * HP + i * DP % HP : i * DP;
        const uint32_t v = vp - cp + c + (uint32_t)r0 * ldx;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? rup : sp, dst, 16, (int)(TP_T || (int)c < left ? v : kOutside),
                                                 TP_T ? 0 : s * 128, 0, 0);
      }
    }
  };

  // ---- fragments of one half step (64 bytes of the reduction)
  const int wq = w / WP, wp = w % WP, g = lane >> 4, l16 = lane & 15;
  // transposed: rows 8 g + l16 / 4 (+ 4 for the second half of a fragment's k) of the half's 32
  const int tz = 8 * g + (l16 >> 2), tsw = 2 * swz_t(tz);
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  auto frag_t = [&](const uint8_t *tile, int rb, int col, int h) -> v4i {
    // col: first of the fragment's 16 columns
    const int c = (col >> 3) + ((l16 & 3) >> 1);
    const uint8_t *p = tile + (32 * h + tz) * rb + 8 * (l16 & 1);
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + ((c ^ tsw) * 16)));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * rb + ((c ^ tsw) * 16)));
    return __builtin_bit_cast(v4i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto frag_q = [&](const uint8_t *tile, int j, int h) -> v4i {
    if (TQ_T) return frag_t(tile, BQ * 2, wq * TQ + 16 * j, h);
    const int r = wq * TQ + 16 * j + l16;
    return *(const v4i *)(tile + r * 128 + (((4 * h + g) ^ swz_r(r)) * 16));
  };
  auto frag_p = [&](const uint8_t *tile, int j, int h) -> v4i {
    if (TP_T) return frag_t(tile, BP * 2, wp * TP + 16 * j, h);
    const int r = wp * TP + 16 * j + l16;
    return *(const v4i *)(tile + r * 128 + (((4 * h + g) ^ swz_r(r)) * 16));
  };

  // ---- scales of 8-bit floating point: a row of x has one a step, so has the tile's
  // part of w (two in a gated block: its branches').  w's are read a step ahead into
  // scalar registers; x's, with the tiles, four steps' at once straight to LDS, as
  // [row][4], or [4][row] from rows of fewer than four, and from there a step ahead.
  // (A load a row and step into registers, 16 lines a quarter wave, took half the
  // kernel's time; read from LDS where they are used, a tenth of what is left.)
  const int kbs = (a.K + kF8Block - 1) / kF8Block;
  static_assert(!F8 || kF8Block % TP == 0, "a wave's columns of one block");
  constexpr int NW8 = F8 && GLU ? 2 : 1, XW = F8 ? (BQ / 64 + NW - 1) / NW : 1;
  const float *sxp[XW];
  const MmConstF *swp[NW8];
  float sw[NW8];
  int sx0 = 0, sxr = 0, xhalf = 0;                              // first block of K last loaded, and read; the latter's half
  const int xstep = kbs >= 4 ? 1 : BQ, xrow = kbs >= 4 ? 4 : 1;
  if constexpr (F8) {
#pragma unroll
    for (int i = 0; i < XW; i++) {
      const int q = (i * NW + w) * 64 + lane;
      const long xr = q < qn ? mm_x_row(a, t.row0 + q) : -1;
      sxp[i] = xr < 0 ? nullptr : a.x_scales + xr * kbs;
    }
    const int nbs = (a.N + kF8Block - 1) / kF8Block;
#pragma unroll
    for (int i = 0; i < NW8; i++) {
      const int b = (p0 + wp * (GLU ? HP : TP)) / kF8Block;
      const long blk = GLU ? ((long)t.e * 2 + (i == 0 ? a.glu.gate0 != 0 : a.glu.up0 != 0)) * nbs + min(b, nbs - 1)
                           : (long)t.e * nbs + min(b, nbs - 1);
      swp[i] = (const MmConstF *)(uintptr_t)a.w_scales + blk * kbs;
    }
  }
  auto load_scales = [&](int s) {
    if constexpr (F8) {
      if (s >= steps || (s > begin && s < sx0 + 4)) return;
      sx0 = kbs < 4 ? 0 : min(s, kbs - 4);
      float *xs = xsl + (s > begin ? (xhalf ^ 1) * BQ * 4 : 0);
#pragma unroll
      for (int i = 0; i < XW; i++) {
        const int r0 = (i * NW + w) * 64;
        if (r0 >= BQ) break;
        if (kbs >= 4) {
          const float *p = sxp[i] ? sxp[i] + sx0 : (const float *)g_mm_zeros;
          __builtin_amdgcn_global_load_lds(p, (lds_void *)(xs + r0 * 4), 16, 0, 0);
        } else {
          for (int k = 0; k < kbs; k++) {
            const float *p = sxp[i] ? sxp[i] + k : (const float *)g_mm_zeros;
            __builtin_amdgcn_global_load_lds(p, (lds_void *)(xs + k * BQ + r0), 4, 0, 0);
          }
        }
      }
    }
  };
  auto load_w = [&](int s) {
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < NW8; i++) sw[i] = swp[i][s];
    }
  };
  float sx[F8 ? NQ : 1];
  auto read_x = [&](int s) {             // (s past the last step: the last)
    if constexpr (F8) {
      s = min(s, steps - 1);
      if (kbs >= 4 && s >= sxr + 4) sxr = sx0, xhalf ^= 1;
      const float *xs = xsl + (wq * TQ + l16) * xrow + xhalf * BQ * 4 + (s - sxr) * xstep;
#pragma unroll
      for (int j = 0; j < NQ; j++) sx[j] = xs[16 * j * xrow];
    }
  };

  typename M::acc acc[NP][NQ];
#pragma unroll
  for (int i = 0; i < NP; i++)
#pragma unroll
    for (int j = 0; j < NQ; j++) acc[i][j] = typename M::acc{0, 0, 0, 0};

  // One stage of LDS: the next step's tiles are loaded once every wave has this
  // one's fragments in registers, and the other blocks of the CU (two or three,
  // by registers and LDS) multiply while they arrive and while this one stores.
  // A second stage in its place leaves room for fewer or smaller blocks and was
  // slower: 16382 x 4096 x 4096 by 2 % (256 x 256, eight waves, one block a CU,
  // which spends a tenth of a tile on its start and end), 32 experts' row gradient
  // by 16 %.
  // Gathered rows' numbers take more registers, so the first half then multiplies
  // before the second is read (weight gradient of 32 groups, 1024 x 6144: 269 us,
  // 295 the other way; int8 prefill 671, 770; rows in order win by up to 5 % with
  // both halves read at once: eight groups of 2048 rows, 4096 x 4096, 529, 558).
  if (begin < steps) {
    gather_rows(begin);
    load(begin);
    load_scales(begin);
    load_w(begin);
    if constexpr (F8) {
      sxr = sx0;
      __builtin_amdgcn_s_waitcnt(0);
      mm_barrier();
      read_x(begin);
      load_scales(begin + 1);
    }
    gather_rows(begin + 1);
  }
  for (int s = begin; s < steps; s++) {
    __builtin_amdgcn_s_waitcnt(0);       // this step's tiles have landed, for every wave
    mm_barrier();
    const uint8_t *lq = lds, *lp = lq + BQ * 128;
    v4i fq[2][NQ], fp[2][NP];
    auto read = [&](int h) {
#pragma unroll
      for (int j = 0; j < NP; j++) fp[h][j] = frag_p(lp, j, h);
#pragma unroll
      for (int j = 0; j < NQ; j++) fq[h][j] = frag_q(lq, j, h);
    };
    auto mul = [&](int h) {
      if constexpr (!F8) {
#pragma unroll
        for (int j = 0; j < NQ; j++)
#pragma unroll
          for (int i = 0; i < NP; i++) acc[i][j] = M::mma(fp[h][i], fq[h][j], acc[i][j]);
      }
    };
    // 8-bit floating point: the operands of a part of the columns at a time, half of them or, where
    // the operands as fp16 fill the registers, a quarter (gated: of one branch)
    MmScale8 zx[F8 ? NQ : 1], zw[NW8];
    constexpr int PARTS8 = TYPE == MM_F8X && NP > 4 ? 4 : 2, HF = NP / PARTS8;
    v8h hq[TYPE == MM_F8X ? NQ : 1][4];
    auto read8 = [&](int b) {
#pragma unroll
      for (int i = 0; i < HF; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) fp[h][b * HF + i] = frag_p(lp, b * HF + i, h);
    };
    auto mul8 = [&](int b) {
      const MmScale8 zb = zw[GLU ? b / (PARTS8 / 2) : 0];
      if constexpr (TYPE == MM_F8) {
        // a block's sums meet the accumulators two instructions later, in the shadow of the
        // ones between; the order is pinned, or more sums are in flight than registers hold
        constexpr int L = 2, CNT = HF * NQ;
        v4f d[L + 1];
        float m[NQ];
#pragma unroll
        for (int j = 0; j < NQ; j++) m[j] = zb.m * zx[j].m;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < CNT + L; c++) {
          if (c < CNT) {
            const int i = b * HF + c / NQ, j = c % NQ;
            d[c % (L + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                join8(fp[0][i], fp[1][i]), join8(fq[0][j], fq[1][j]), v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, zb.code, 0, zx[j].code);
          }
          if (c >= L) {
            const int o = c - L, i = b * HF + o / NQ, j = o % NQ;
#pragma unroll
            for (int k = 0; k < 4; k++) acc[i][j][k] = fmaf(d[o % (L + 1)][k], m[j], acc[i][j][k]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else if constexpr (F8) {
        // the block's sums of a fragment of w and all of x's, then their scales in two factors
        // (mm_factors8), one product and one fused addition a sum
        float f1[NQ], f2[NQ];
#pragma unroll
        for (int j = 0; j < NQ; j++) mm_factors8(zb, zx[j], f1[j], f2[j]);
#pragma unroll
        for (int i = b * HF; i < b * HF + HF; i++) {
          v4f d[NQ];
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const v8h hp = codes_f16(fp[c >> 1][i][2 * (c & 1)], fp[c >> 1][i][2 * (c & 1) + 1]);
#pragma unroll
            for (int j = 0; j < NQ; j++) d[j] = mfma_f16(hp, hq[j][c], c ? d[j] : v4f{0.f, 0.f, 0.f, 0.f});
          }
#pragma unroll
          for (int j = 0; j < NQ; j++)
#pragma unroll
            for (int k = 0; k < 4; k++) acc[i][j][k] = fmaf(d[j][k] * f1[j], f2[j], acc[i][j][k]);
        }
      }
    };
    if constexpr (F8) {
#pragma unroll
      for (int j = 0; j < NQ; j++) {
        zx[j] = mm_scale8(sx[j]);
#pragma unroll
        for (int h = 0; h < 2; h++) fq[h][j] = frag_q(lq, j, h);
      }
#pragma unroll
      for (int i = 0; i < NW8; i++) zw[i] = mm_scale8(sw[i]);
      read8(0);
      read_x(s + 1);
      if constexpr (TYPE == MM_F8X) {
#pragma unroll
        for (int j = 0; j < NQ; j++)
#pragma unroll
          for (int c = 0; c < 4; c++) hq[j][c] = codes_f16(fq[c >> 1][j][2 * (c & 1)], fq[c >> 1][j][2 * (c & 1) + 1]);
      }
#pragma unroll
      for (int b = 0; b + 1 < PARTS8; b++) {
        mul8(b);
        // (kept in front of the next part's reads and the branch below: sunk past them, more
        // parts' operands would be live and the accumulators spill)
#pragma unroll
        for (int i = b * HF; i < b * HF + HF; i++)
#pragma unroll
          for (int j = 0; j < NQ; j++) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
        read8(b + 1);
      }
    } else {
      read(0);
      if (GATHER && !NEAR) {
        mul(0);
        __builtin_amdgcn_sched_barrier(0);
      }
      read(1);
    }
    if (s + 1 < steps) {
      wait_lgkm0();                      // the stage is free once every wave has read it
      mm_barrier();
      load(s + 1);
      load_w(s + 1);
      load_scales(s + 2);
      gather_rows(s + 2);
    }
    if constexpr (F8) {
      mul8(PARTS8 - 1);
    } else {
      if (!GATHER || NEAR) mul(0);
      mul(1);
    }
  }

  // ---- outputs
  const long orow = OP == MM_DW ? (long)t.e * a.N + q0 : (long)t.row0;   // row 0 of the tile
  MmScale xs[TYPE == MM_I8 ? NQ : 1];
  if constexpr (TYPE == MM_I8) {
#pragma unroll
    for (int j = 0; j < NQ; j++) {
      const int q = wq * TQ + 16 * j + l16;
      const long xr = q < qn ? mm_x_row(a, t.row0 + q) : -1;
      xs[j] = mm_scale(xr < 0 ? 0.f : a.x_scales[xr]);
    }
  }
  // Sixteen rows of 64 columns at a time go through the wave's own part of LDS, so
  // that a store writes whole rows of them (four of 256 bytes, eight of 128): 16
  // bytes of each of 16 rows in every quarter wave, as the accumulators lie, cost
  // a fp32 weight gradient of 64 x 7168 x 576 328 us for 195 us (5.4 TB/s), one in
  // 16 bits 150 for 122.  Weight gradients, which are read much later, are stored
  // past the caches: another 210 -> 195 us and 122 -> 87 us there; the other
  // products' rows, which the next kernel reads, gain 0 to 3 % and stay.
  wait_lgkm0();                          // every wave has read its last fragments
  mm_barrier();
  uint8_t *mine = lds + w * kOutStage;
  auto fence = [] {                      // LDS accesses of a wave are in order: for the compiler only
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  };
  if constexpr (GLU) {
    constexpr int NG = NP / 2;           // fragments of a branch
    // v(i, k): result k of fragment i, to columns col + 16 i .. of rows of ld; what lies in the
    // tile goes to o(row, column, data)
    auto rows_out = [&](auto wide, int j, auto v, auto o) {
      constexpr int WB = decltype(wide)::value, RB = NG * 16 * WB + 16, LR = NG * WB, CW = 16 / WB;
      fence();
#pragma unroll
      for (int i = 0; i < NG; i++) {
        uint8_t *d = mine + l16 * RB + (16 * i + 4 * g) * WB;
        if constexpr (WB == 4) *(v4f *)d = v4f{v(i, 0), v(i, 1), v(i, 2), v(i, 3)};
        else *(v2u *)d = v2u{v(i, 0), v(i, 2)};   // two results at once
      }
      fence();
#pragma unroll
      for (int r = 0; r < 16; r += 64 / LR) {
        const int row = r + lane / LR, q = wq * TQ + 16 * j + row, c = p0 + wp * HP + CW * (lane % LR);
        const v4i d = *(const v4i *)(mine + row * RB + (lane % LR) * 16);
        if (row < 16 && q < qn && c < pn) o((long)t.row0 + q, c, d);
      }
    };
    if (a.splits > 1 || parts > 1) {
      // [gate, up][row][column] of a tile's part, or the rows' columns as w has them
      const bool tile = parts > 1;
      float *sum = a.part + (tile ? ((long)tail_at * parts + part) * BQ * BP : (long)blockIdx.y * a.R * 2 * pn);
#pragma unroll
      for (int j = 0; j < NQ; j++)
#pragma unroll
        for (int b = 0; b < 2; b++) {
          const int c0 = b ? a.glu.up0 : a.glu.gate0;
          rows_out(MmConst<4>{}, j, [&](int i, int k) { return acc[b * NG + i][j][k]; }, [&](long r, int c, v4i d) {
            *(v4i *)(sum + (tile ? (long)((b * BQ + (int)(r - t.row0)) * BC + c - p0) : r * 2 * pn + c0 + c)) = d;
          });
        }
      return;
    }
    if constexpr (!F8) {
      if (a.pre_out) {
        // kept in the operands' type for the backward pass; h below is of the unrounded sums
#pragma unroll
        for (int j = 0; j < NQ; j++)
#pragma unroll
          for (int b = 0; b < 2; b++) {
            const int c0 = b ? a.glu.up0 : a.glu.gate0;
            rows_out(MmConst<2>{}, j, [&](int i, int k) { return mm_pack<TYPE>(acc[b * NG + i][j][k], acc[b * NG + i][j][k + 1]); },
                     [&](long r, int c, v4i d) { *(v4i *)((uint16_t *)a.pre_out + r * 2 * pn + c0 + c) = d; });
          }
      }
    }
#pragma unroll
    for (int i = 0; i < NG; i++)
#pragma unroll
      for (int j = 0; j < NQ; j++)
#pragma unroll
        for (int k = 0; k < 4; k++) acc[i][j][k] = glu_act(acc[i][j][k], acc[NG + i][j][k], a.glu);
    mm_by_output<TYPE>(a.out_type, [&](auto out) {
      constexpr int OUT = decltype(out)::value;
      if constexpr (OUT != MM_PART) {
#pragma unroll
        for (int j = 0; j < NQ; j++) {
          if constexpr (OUT == MM_FP32)
            rows_out(MmConst<4>{}, j, [&](int i, int k) { return acc[i][j][k]; },
                     [&](long r, int c, v4i d) { *(v4i *)((float *)a.out + r * pn + c) = d; });
          else
            rows_out(MmConst<2>{}, j, [&](int i, int k) { return mm_pack<OUT>(acc[i][j][k], acc[i][j][k + 1]); },
                     [&](long r, int c, v4i d) { *(v4i *)((uint16_t *)a.out + r * pn + c) = d; });
        }
      }
    });
    return;
  }
  if constexpr (OP == MM_GLU_DX) if (a.splits <= 1 && parts <= 1) {
    // 16 rows of 64 columns of dh, eight columns a lane, with the projections there
    constexpr int RB = 64 * 4 + 16;
#pragma unroll
    for (int i0 = 0; i0 < NP; i0 += 4)
#pragma unroll
      for (int j = 0; j < NQ; j++) {
        fence();
#pragma unroll
        for (int i = 0; i < 4; i++) *(v4f *)(mine + l16 * RB + (16 * i + 4 * g) * 4) = __builtin_bit_cast(v4f, acc[i0 + i][j]);
        fence();
#pragma unroll
        for (int r = 0; r < 16; r += 8) {
          const int row = r + lane / 8, q = wq * TQ + 16 * j + row, c = p0 + wp * TP + 16 * i0 + 8 * (lane % 8);
          const uint8_t *d = mine + row * RB + (lane % 8) * 32;
          const v4f d0 = *(const v4f *)d, d1 = *(const v4f *)(d + 16);
          if (q < qn && c < pn) glu_back8<TYPE>(a.glu, pn, a.pre, a.out, a.h, (long)t.row0 + q, c, d0, d1);
        }
      }
    return;
  }
  mm_by_output<TYPE>(a.splits > 1 || parts > 1 ? MM_PART : a.out_type, [&](auto out) {
    constexpr int OUT = decltype(out)::value;
    constexpr bool WIDE = OUT == MM_FP32 || OUT == MM_PART, NT = OP == MM_DW && OUT != MM_PART;
    constexpr int RB = WIDE ? 64 * 4 + 16 : 64 * 2 + 16;   // a row, and 16 bytes that spread the rows over the banks
    constexpr int LR = WIDE ? 16 : 8, CW = 64 / LR;        // lanes a row, columns a lane
    const long outs = OP == MM_DW ? (long)a.E * a.N : (long)a.R;
    float *sums = a.part + (OUT == MM_PART && parts <= 1 ? (long)blockIdx.y * outs * pn : 0);
#pragma unroll
    for (int i0 = 0; i0 < NP; i0 += 4) {
      const int pc = p0 + wp * TP + 16 * i0, po = pc + CW * (lane % LR);
      MmScale ws[TYPE == MM_I8 ? 16 : 1];
      if constexpr (TYPE == MM_I8) {
#pragma unroll
        for (int k = 0; k < 16; k++) {
          const int p = pc + 16 * (k >> 2) + 4 * g + (k & 3);
          ws[k] = mm_scale(p < pn ? a.w_scales[(size_t)t.e * a.N + p] : 0.f);
        }
      }
#pragma unroll
      for (int j = 0; j < NQ; j++) {
        fence();
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const auto e = acc[i0 + i][j][k];
            if constexpr (OUT == MM_PART) v[k] = __builtin_bit_cast(float, e);
            else if constexpr (TYPE == MM_I8) v[k] = mm_scaled(e, xs[j], ws[4 * i + k]);
            else v[k] = e;
          }
          uint8_t *o = mine + l16 * RB + (16 * i + 4 * g) * (WIDE ? 4 : 2);
          if constexpr (WIDE) *(v4f *)o = v4f{v[0], v[1], v[2], v[3]};
          else *(v2u *)o = v2u{mm_pack<OUT>(v[0], v[1]), mm_pack<OUT>(v[2], v[3])};
        }
        fence();
#pragma unroll
        for (int r = 0; r < 16; r += 64 / LR) {
          const int row = r + lane / LR, q = wq * TQ + 16 * j + row;
          const v4i d = *(const v4i *)(mine + row * RB + (lane % LR) * 16);
          if (q >= qn || po >= pn) continue;
          const long at = (orow + q) * pn + po;
          if constexpr (OUT == MM_PART) *(v4i *)(sums + (parts > 1 ? ((long)tail_at * parts + part) * BQ * BP + q * BP + po - p0 : at)) = d;
          else if constexpr (OUT == MM_FP32) mm_store_f32<NT>(a, at, __builtin_bit_cast(v4f, d));
          else mm_store<NT>((v4i *)((uint16_t *)a.out + at), d);
        }
      }
    }
  });
}

// Joins the parts of a split reduction, in their order: a block per output row,
// eight columns a thread at a time.  A row of the groups' rows finds its group
// by comparing all offsets; rows in no group are left alone.
template <int TYPE>
__global__ __launch_bounds__(256) void k_mm_join(MmArgs a) {
  typedef typename MmElem<TYPE>::acc Acc;
  const int pn = a.op == MM_FORWARD ? a.N : a.K;
  const long row = blockIdx.x, outs = a.op == MM_DW ? (long)a.E * a.N : (long)a.R;
  int e = 0;
  if (a.op != MM_DW && a.first) {
    const int lane = threadIdx.x & 63;
    e = -1;
    for (int b = 0; b < a.E; b += 64) {
      int lo = 0, hi = 0;
      if (b + lane < a.E) mm_group(a, b + lane, lo, hi);
      const unsigned long long m = __ballot(row >= lo && row < hi);
      if (m) {
        e = b + __ffsll(m) - 1;
        break;
      }
    }
    if (e < 0) return;
  }
  if (a.accumulate) {                    // of a weight gradient: a group without rows has no parts
    int lo, hi;
    mm_group(a, (int)(row / a.N), lo, hi);
    if (lo == hi) return;
  }
  MmScale xs = {0.f, 0};
  if (TYPE == MM_I8) {
    const long xr = mm_x_row(a, (int)row);
    if (xr >= 0) xs = mm_scale(a.x_scales[xr]);
  }
  mm_by_output<TYPE>(a.out_type, [&](auto out) {
    constexpr int OUT = decltype(out)::value;
    if constexpr (OUT != MM_PART) {
      for (int p = threadIdx.x * 8; p < pn; p += 256 * 8) {
        Acc s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        for (int i = 0; i < a.splits; i++) {
          const Acc *part = (const Acc *)(a.part + ((long)i * outs + row) * pn + p);
          s[0] += part[0];
          s[1] += part[1];
        }
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const auto sum = s[k >> 2][k & 3];
          if constexpr (TYPE == MM_I8) v[k] = mm_scaled(sum, xs, mm_scale(a.w_scales[(size_t)e * a.N + p + k]));
          else v[k] = sum;
        }
        mm_store8<OUT>(a, row * pn + p, v);
      }
    }
  });
}

// Eight columns from p of row `row` out of their joined sums, sum(b, s) for branch b (gate,
// up) or of the only one: as they are, through the activation, or dh through its gradient.
template <int OP, int TYPE, typename Sum>
__device__ __forceinline__ void glu_finish(const MmArgs &a, int pn, long row, int p, Sum sum) {
  v4f s[2][2];
  sum(0, s[0]);
  if constexpr (OP == MM_GLU_DX) {
    glu_back8<TYPE>(a.glu, pn, a.pre, a.out, a.h, row, p, s[0][0], s[0][1]);
  } else {
    float v[8];
    if constexpr (OP == MM_GLU) {
      sum(1, s[1]);
      if constexpr (TYPE == MM_BF16 || TYPE == MM_FP16) {
        if (a.pre_out) {
#pragma unroll
          for (int b = 0; b < 2; b++)
            *(v4i *)((uint16_t *)a.pre_out + row * 2 * pn + (b ? a.glu.up0 : a.glu.gate0) + p) =
                v4i{(int)mm_pack<TYPE>(s[b][0][0], s[b][0][1]), (int)mm_pack<TYPE>(s[b][0][2], s[b][0][3]),
                    (int)mm_pack<TYPE>(s[b][1][0], s[b][1][1]), (int)mm_pack<TYPE>(s[b][1][2], s[b][1][3])};
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; k++) {
      if constexpr (OP == MM_GLU) v[k] = glu_act(s[0][k >> 2][k & 3], s[1][k >> 2][k & 3], a.glu);
      else v[k] = s[0][k >> 2][k & 3];
    }
    mm_by_output<TYPE>(a.out_type, [&](auto out) {
      constexpr int OUT = decltype(out)::value;
      if constexpr (OUT != MM_PART) mm_store8<OUT>(a, row * pn + p, v);
    });
  }
}

// The same for the gated block: the parts of both projections, then the activation,
// or the parts of dh, then its gradient.
template <int OP, int TYPE>
__global__ __launch_bounds__(256) void k_glu_join(MmArgs a) {
  const int pn = mm_outs(OP, a.N, a.K), wide = OP == MM_GLU ? 2 * pn : pn;
  const long row = blockIdx.x;
  if (a.first) {                         // rows in no group are left alone
    const int lane = threadIdx.x & 63;
    bool in = false;
    for (int b = 0; b < a.E && !in; b += 64) {
      int lo = 0, hi = 0;
      if (b + lane < a.E) mm_group(a, b + lane, lo, hi);
      in = __any(row >= lo && row < hi);
    }
    if (!in) return;
  }
  for (int p = threadIdx.x * 8; p < pn; p += 256 * 8)
    glu_finish<OP, TYPE>(a, pn, row, p, [&](int b, v4f *s) {
      const int c = OP != MM_GLU ? p : p + (b ? a.glu.up0 : a.glu.gate0);
      s[0] = s[1] = v4f{0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i < a.splits; i++) {
        const v4f *part = (const v4f *)(a.part + ((long)i * a.R + row) * wide + c);
        s[0] += part[0];
        s[1] += part[1];
      }
    });
}

// Joins the parts of the last round's tiles: a block per tile and what rows of it 256
// threads have at eight columns each.
template <int OP, int TYPE, int BQ, int BP, int MINW>
__global__ __launch_bounds__(256) void k_tail_join(MmArgs a) {
  constexpr int BC = mm_tile_cols(OP, BP), TR = BC / 8, ES = sizeof(typename MmElem<TYPE>::t);
  const int pn = mm_outs(OP, a.N, a.K), ptiles = (pn + BC - 1) / BC;
  const int reduction = mm_forward(OP) ? a.K : a.N, all = (reduction + 128 / ES - 1) / (128 / ES);
  MmTile t;
  int parts = 1;
  const int at = (int)blockIdx.x;
  if (!mm_tile_by<BQ>(a, ptiles, t, [&](int nt) {
        const MmTail m = mm_tail(nt, 256 * MINW, all);
        parts = m.parts;
        return at < m.rem ? m.full + at : -1;
      }))
    return;
  const float *tile = a.part + (long)at * parts * BQ * BP;
  const int c = (int)threadIdx.x % TR * 8, p = t.pt * BC + c;
  if (p >= pn) return;
  const int q = (int)blockIdx.y * (256 / TR) + (int)threadIdx.x / TR;
  if (q >= t.rows) return;
  glu_finish<OP, TYPE>(a, pn, (long)t.row0 + q, p, [&](int b, v4f *s) {
    const float *v = tile + (b * BQ + q) * BC + c;
    s[0] = s[1] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < parts; i++) {
      s[0] += *(const v4f *)(v + (long)i * BQ * BP);
      s[1] += *(const v4f *)(v + (long)i * BQ * BP + 4);
    }
  });
}

template <int OP, int TYPE, int BQ, int BP, int WQ, int WP, int MINW>
static hipError_t launch_tile(const MmArgs &a, hipStream_t s) {
  constexpr bool TAIL = mm_has_tail(OP, TYPE, BQ, BP);
  constexpr int BC = mm_tile_cols(OP, BP);
  const long pn = mm_outs(OP, a.N, a.K), ptiles = (pn + BC - 1) / BC;
  long blocks;
  if (OP == MM_DW) blocks = 8l * a.E * (((a.N + BQ - 1) / BQ * ptiles + 7) / 8);
  else blocks = (((a.R + BQ - 1) / BQ + (a.first ? (a.E < a.R ? a.E : a.R) : 0)) * ptiles + 7) / 8 * 8;
  const long slots = 256 * MINW;
  if (TAIL && a.tail) blocks += slots;   // the last round's parts
  if (blocks > INT32_MAX / (64 * WQ * WP)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks, (unsigned)a.splits), threads(64 * WQ * WP);
  // (row gradients have no gathered rows)
  if (!mm_dx(OP) && a.rows) hipLaunchKernelGGL((k_mm_tile<OP, TYPE, BQ, BP, WQ, WP, !mm_dx(OP), MINW>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((k_mm_tile<OP, TYPE, BQ, BP, WQ, WP, false, MINW>), grid, threads, 0, s, a);
  if constexpr (TAIL) {
    if (a.tail) hipLaunchKernelGGL((k_tail_join<OP, TYPE, BQ, BP, MINW>), dim3((unsigned)(slots / 2), BQ * BC / 2048), dim3(256), 0, s, a);
  }
  if (a.splits > 1) {
    const long outs = OP == MM_DW ? (long)a.E * a.N : (long)a.R;
    if constexpr (OP == MM_GLU || OP == MM_GLU_DX) hipLaunchKernelGGL((k_glu_join<OP, TYPE>), dim3((unsigned)outs), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(k_mm_join<TYPE>, dim3((unsigned)outs), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

// ------------------------------------------------------------ few rows a group
//
// Weights streamed once: a block takes up to 16 rows of a group and 16
// channels, its waves the 128-byte columns of the reduction in turn.  Each wave
// runs a ring of kStreamSlots columns of its own in LDS, loaded straight from
// memory in whole 128-byte lines (8 rows a load), so it needs no barrier until
// the waves' sums meet in wave order.  Loading MFMA operands into registers
// instead touches 16 rows in every 16 lanes: 33 MB of int8 weights in 13.1 us
// against 7.7 us this way (4.3 TB/s), 48 experts' bf16 rows (0.79 GB) in 133 us
// against 129 us (5.8 TB/s).  Four waves of two slots leave four blocks a CU:
// deeper rings or more waves measured 130 to 154 us and 8.6 to 13 us.
constexpr int kStreamSlots = 2, kStreamWaves = 4;

// The 16 x 16 MFMA operands of one column: weights at LDS offset pw, rows of x
// at px, both halves of the reduction.  Read and waited for in one statement,
// so the loads in flight to the other slots are not waited for.
__device__ __forceinline__ void stream_read(uint32_t pw0, uint32_t pw1, uint32_t px0, uint32_t px1, v4i *w, v4i *x) {
  asm volatile(
      "ds_read_b128 %0, %4\n"
      "ds_read_b128 %1, %5\n"
      "ds_read_b128 %2, %6\n"
      "ds_read_b128 %3, %7\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(w[0]), "=&v"(w[1]), "=&v"(x[0]), "=&v"(x[1])
      : "v"(pw0), "v"(pw1), "v"(px0), "v"(px1)
      : "memory");
}

// The same with a column's two scales.
__device__ __forceinline__ void stream_read8(uint32_t pw0, uint32_t pw1, uint32_t px0, uint32_t px1, uint32_t s0,
                                             uint32_t s1, v4i *w, v4i *x, float &a, float &b) {
  asm volatile(
      "ds_read_b128 %0, %6\n"
      "ds_read_b128 %1, %7\n"
      "ds_read_b128 %2, %8\n"
      "ds_read_b128 %3, %9\n"
      "ds_read_b32 %4, %10\n"
      "ds_read_b32 %5, %11\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(w[0]), "=&v"(w[1]), "=&v"(x[0]), "=&v"(x[1]), "=&v"(a), "=&v"(b)
      : "v"(pw0), "v"(pw1), "v"(px0), "v"(px1), "v"(s0), "v"(s1)
      : "memory");
}

// A gated block's 16 channels are eight of the gate and the same eight of the up branch.
template <int OP, int TYPE, bool GATHER>
__global__ __launch_bounds__(64 * kStreamWaves) void k_mm_stream(MmArgs a) {
  typedef MmElem<TYPE> M;
  typedef typename M::acc Acc;
  constexpr int ES = sizeof(typename M::t), D = kStreamSlots, NW = kStreamWaves;
  constexpr bool GLU = OP == MM_GLU, F8 = TYPE == MM_F8X;
  constexpr int kSlot = 4096 + (F8 ? 256 : 0);   // 16 weight rows, 16 rows of x, scales
  constexpr int RS = 16 + 4;             // a row of sums, padded so that rows start on other banks
  __shared__ __align__(1024) uint8_t ring[NW][D][kSlot];
  __shared__ Acc sum[NW * 16 * RS / 4];
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  constexpr int PC = mm_tile_cols(OP, 16);   // columns of the output a block has
  MmTile t;
  if (!mm_find_tile<16>(a, (a.N + PC - 1) / PC, t)) return;
  const int p0 = t.pt * PC, l16 = lane & 15, g = lane >> 4;
  const uint32_t ld = (uint32_t)a.K * ES;
  const int units = (int)((ld + 127) >> 7);
  const uint8_t *we = (const uint8_t *)a.w + (size_t)t.e * (GLU ? 2 * a.N : a.N) * ld;
  const Rsrc wb = mm_rsrc(we + (size_t)(p0 + (GLU ? a.glu.gate0 : 0)) * ld, (uint32_t)min(PC, a.N - p0) * ld);
  const Rsrc wup = GLU ? mm_rsrc(we + (size_t)(p0 + a.glu.up0) * ld, (uint32_t)min(PC, a.N - p0) * ld) : wb;
  // loads: row 8 i + lane / 8, its chunk swizzled as in the tile kernels
  uint32_t vw[2], ck[2];
  const uint8_t *xp[2];
  bool live[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int r = 8 * i + (lane >> 3);
    ck[i] = (uint32_t)((lane & 7) ^ swz_r(r)) * 16;
    vw[i] = (uint32_t)(GLU ? lane >> 3 : r) * ld + ck[i];   // (gated: load 1 is of the up branch)
    const long xr = r < t.rows ? (GATHER ? mm_x_row(a, t.row0 + r) : (long)t.row0 + r) : -1;
    live[i] = xr >= 0;
    xp[i] = (const uint8_t *)a.x + (live[i] ? (size_t)xr * ld : 0) + ck[i];
  }
  // this thread's outputs after the join: four channels of one row, and their scales
  const int oq = threadIdx.x / (PC / 4), op = threadIdx.x % (PC / 4) * 4;
  const bool writes = oq < t.rows && p0 + op < a.N;   // (which leaves 16 or, gated, 8 columns to 64 or 32 threads)
  float xs = 0.f;
  v4f ws = {0.f, 0.f, 0.f, 0.f};
  if (TYPE == MM_I8 && writes) {
    const long xr = mm_x_row(a, t.row0 + oq);
    if (xr >= 0) xs = a.x_scales[xr];
#pragma unroll
    for (int k = 0; k < 4; k++) ws[k] = a.w_scales[(size_t)t.e * a.N + p0 + op + k];
  }
  const uint32_t base = (uint32_t)(uintptr_t)(lds_void *)&ring[w][0][0];
  const uint32_t rd0 = base + l16 * 128 + ((g ^ swz_r(l16)) * 16), rd1 = base + l16 * 128 + (((4 + g) ^ swz_r(l16)) * 16);
  Acc acc = {0, 0, 0, 0};
  const int n = (units - w + NW - 1) / NW;   // columns of this wave
  // 8-bit floating point: a column of the reduction is a block of one scale.  One more load
  // brings a column's: lanes 0 to 15 those of the rows of x, 16 and 17 w's (gated: the
  // gate's and the up branch's), the others zeros.
  const float *sp = (const float *)g_mm_zeros;
  int sstep = 0;                         // floats a column
  if constexpr (F8) {
    const int nbs = (a.N + kF8Block - 1) / kF8Block, b = p0 / kF8Block;
    if (lane < 16) {
      const long xr = lane < t.rows ? (GATHER ? mm_x_row(a, t.row0 + lane) : (long)t.row0 + lane) : -1;
      if (xr >= 0) sp = a.x_scales + xr * units, sstep = 1;
    } else if (lane < 18) {
      const long half = GLU ? (long)t.e * 2 + ((lane == 17 ? a.glu.up0 : a.glu.gate0) != 0) : (long)t.e;
      sp = a.w_scales + (half * nbs + b) * units, sstep = 1;
    }
  }

  // XI: loads of eight rows of x a column
  auto body = [&](auto xi) {
    constexpr int XI = decltype(xi)::value, CNT = 2 + XI + F8;
    auto load = [&](int s) {
      const uint32_t k = (uint32_t)(s * NW + w) * 128;
      uint8_t *dst = &ring[w][s % D][0];
#pragma unroll
      for (int i = 0; i < 2; i++)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(i ? wup : wb, (lds_void *)(dst + i * 1024), 16,
                                                 (int)(k + ck[i] < ld ? vw[i] : kOutside), (int)k, 0, 0);
#pragma unroll
      for (int i = 0; i < XI; i++) {
        const uint8_t *p = live[i] && k + ck[i] < ld ? xp[i] + k : (const uint8_t *)g_mm_zeros;
        __builtin_amdgcn_global_load_lds(p, (lds_void *)(dst + 2048 + i * 1024), 16, 0, 0);
      }
      if constexpr (F8) __builtin_amdgcn_global_load_lds(sp + (s * NW + w) * sstep, (lds_void *)(dst + 4096), 4, 0, 0);
    };
    for (int s = 0; s < min(n, D - 1); s++) load(s);
    for (int s = 0; s < n; s++) {
      if (s + D - 1 < n) {
        load(s + D - 1);                 // into the slot read in the step before
        wait_vm<(D - 1) * CNT>();
      } else {
        wait_vm<0>();
      }
      const uint32_t o = (uint32_t)(s % D) * kSlot;
      v4i fw[2], fx[2];
      if constexpr (F8) {
        // the scale of w that the sums of lane group g have
        float sc, sx;
        stream_read8(rd0 + o, rd1 + o, rd0 + o + 2048, rd1 + o + 2048, base + o + 4096 + (GLU && g >= 2 ? 68 : 64),
                     base + o + 4096 + l16 * 4, fw, fx, sc, sx);
        acc = f8_block(acc, join8(fw[0], fw[1]), join8(fx[0], fx[1]), mm_scale8(sc), mm_scale8(sx));
      } else {
        stream_read(rd0 + o, rd1 + o, rd0 + o + 2048, rd1 + o + 2048, fw, fx);
        acc = M::mma(fw[0], fx[0], acc);
        acc = M::mma(fw[1], fx[1], acc);
      }
    }
  };
  // rows past XI * 8 of x are not loaded: their MFMA columns hold what LDS held and are not stored
  if (t.rows <= 8) body(MmConst<1>{});
  else body(MmConst<2>{});
  // sums of the waves: [wave][row][channel]
  sum[((w * 16 + l16) * RS + 4 * g) >> 2] = acc;
  __syncthreads();
  mm_by_output<TYPE>(a.out_type, [&](auto out) {
    constexpr int OUT = decltype(out)::value;
    if (!writes) return;
    auto joined = [&](int c) {
      Acc r = sum[(oq * RS + c) >> 2];
#pragma unroll
      for (int v = 1; v < NW; v++) r += sum[((v * 16 + oq) * RS + c) >> 2];
      return r;
    };
    const Acc r = joined(op);
    Acc up = r;
    if constexpr (GLU) {
      up = joined(8 + op);
      if constexpr (!F8) {
        if (a.pre_out) {
          v2u *o = (v2u *)((uint16_t *)a.pre_out + (long)(t.row0 + oq) * 2 * a.N + p0 + op);
          *(v2u *)((uint16_t *)o + a.glu.gate0) = v2u{mm_pack<TYPE>(r[0], r[1]), mm_pack<TYPE>(r[2], r[3])};
          *(v2u *)((uint16_t *)o + a.glu.up0) = v2u{mm_pack<TYPE>(up[0], up[1]), mm_pack<TYPE>(up[2], up[3])};
        }
      }
    }
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      if constexpr (GLU) v[k] = glu_act(r[k], up[k], a.glu);
      else if constexpr (TYPE == MM_I8) v[k] = mm_scaled(r[k], mm_scale(xs), mm_scale(ws[k]));
      else v[k] = r[k];
    }
    mm_store4<OUT>(a, (long)(t.row0 + oq) * a.N + p0 + op, v);
  });
}

template <int OP, int TYPE>
static hipError_t launch_stream(const MmArgs &a, hipStream_t s) {
  constexpr int PC = mm_tile_cols(OP, 16);
  const long tiles = (a.R + 15) / 16 + (a.first ? (a.E < a.R ? a.E : a.R) : 0);
  const long blocks = (tiles * ((a.N + PC - 1) / PC) + 7) / 8 * 8;
  if (a.rows) hipLaunchKernelGGL((k_mm_stream<OP, TYPE, true>), dim3((unsigned)blocks), dim3(64 * kStreamWaves), 0, s, a);
  else hipLaunchKernelGGL((k_mm_stream<OP, TYPE, false>), dim3((unsigned)blocks), dim3(64 * kStreamWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
