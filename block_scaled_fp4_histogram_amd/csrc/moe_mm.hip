// Ragged expert products for gfx950: forward, row gradient and weight gradient
// over 16-bit operands, and the forward product over 8-bit integers.
#include "moe_device.h"
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

// f(integral constant of the output type): the branch on it stands outside the stores.
template <int V>
struct MmConst {
  static constexpr int value = V;
};
constexpr int MM_PART = 5;   // 32-bit sums of one part of the reduction, as they are
template <typename F>
__device__ __forceinline__ void mm_by_output(int out_type, F f) {
  if (out_type == MM_PART) f(MmConst<MM_PART>{});
  else if (out_type == MM_FP32) f(MmConst<MM_FP32>{});
  else if (out_type == MM_BF16) f(MmConst<MM_BF16>{});
  else f(MmConst<MM_FP16>{});
}

// ------------------------------------------------------------ tile kernels

typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr uint32_t kOutside = 0x80000000u;   // lane offset past every resource: loads zeros

// A gathered row that names no row of x, and the part of a row past its end,
// are read from here.
__device__ const uint32_t g_mm_zeros[4] = {0, 0, 0, 0};

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

template <int BQ>
__device__ __forceinline__ bool mm_find_tile(const MmArgs &a, int ptiles, MmTile &t) {
  const int lane = threadIdx.x & 63;
  if (!a.first) {                        // one group: the same order without the scans
    const int total = (a.R + BQ - 1) / BQ, nt = total * ptiles, chunk = (nt + 7) >> 3;
    const int id = ((int)blockIdx.x & 7) * chunk + ((int)blockIdx.x >> 3);
    if (((int)blockIdx.x >> 3) >= chunk || id >= nt) return false;
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
  const int total = uniform(__shfl(sum, 63)), nt = total * ptiles;
  const int chunk = (nt + 7) >> 3, b = (int)blockIdx.x;
  const int id = (b & 7) * chunk + (b >> 3);
  // (a total below zero: offsets that fall, whose groups overlap past 2^31 tiles)
  if (total <= 0 || (b >> 3) >= chunk || id >= nt) return false;
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
  constexpr bool TQ_T = OP == MM_DW, TP_T = OP != MM_FORWARD;   // transposed operands
  constexpr int TQ = BQ / WQ, TP = BP / WP, NQ = TQ / 16, NP = TP / 16;
  constexpr int CQ = BQ / 8 / NW, CP = BP / 8 / NW;             // loads of 1 KB a wave and step
  constexpr int kStage = (BQ + BP) * 128;
  static_assert(TP % 64 == 0 && TQ % 16 == 0 && CQ >= 1 && CP >= 1, "tile shape");
  static_assert(!TQ_T || (BQ % 128 == 0 && TQ % 64 == 0), "transposed Q");
  static_assert(!TP_T || BP % 128 == 0, "transposed P");
  constexpr int kOutStage = 16 * (64 * 4 + 16);                 // of one wave, for its outputs
  static_assert(NW * kOutStage <= kStage, "outputs through LDS");
  __shared__ __align__(1024) uint8_t lds[kStage];

  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int pn = OP == MM_FORWARD ? a.N : a.K;                  // output columns
  const int ptiles = (pn + BP - 1) / BP;
  MmTile t;
  int q0 = 0, qn, zn;                                           // output rows of the tile, reduction
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
    if (!mm_find_tile<BQ>(a, ptiles, t)) return;
    qn = t.rows;
    zn = OP == MM_FORWARD ? a.K : a.N;
  }
  const int p0 = t.pt * BP;
  constexpr int ZS = (TQ_T || TP_T) ? 64 : 128 / ES;            // reduction elements a step
  // with a split reduction, this block's share of the steps
  const int all = (zn + ZS - 1) / ZS, share = a.splits > 1 ? (all + a.splits - 1) / a.splits : all;
  const int begin = (int)blockIdx.y * share, steps = min(all, begin + share);

  // ---- loads of one step
  const uint8_t *x = (const uint8_t *)a.x, *dy = (const uint8_t *)a.dy;
  const uint8_t *wt = (const uint8_t *)a.w + (size_t)t.e * a.N * a.K * ES;
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
  const uint32_t ldq = OP == MM_FORWARD ? ldx : ldy;
  const uint32_t vq = (uint32_t)rq0 * ldq + cq, vp = (uint32_t)rp0 * ldx + cp;
  const Rsrc rq = OP == MM_FORWARD  ? mm_rsrc(x + (GATHER ? 0 : (size_t)t.row0 * ldx), (uint32_t)qn * ldx)
                  : OP == MM_DX     ? mm_rsrc(dy + (size_t)t.row0 * ldy, (uint32_t)qn * ldy)
                                    : mm_rsrc(dy, 0);
  const Rsrc rp = OP == MM_FORWARD ? mm_rsrc(wt + (size_t)p0 * ldx, (uint32_t)min(BP, pn - p0) * ldx) : mm_rsrc(wt, 0);
  // forward gather: each load's row of x
  constexpr bool GF = GATHER && OP == MM_FORWARD, GW = GATHER && OP == MM_DW;
  int grow[GF ? CQ : 1];
  if constexpr (GF) {
#pragma unroll
    for (int i = 0; i < CQ; i++) {
      const int r = rq0 + i * DQ;
      grow[i] = r < qn ? (int)mm_x_row(a, t.row0 + r) : -1;
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
    const Rsrc sp = OP == MM_DX   ? mm_rsrc(wt + (size_t)(s * ZS) * ldx, zleft * ldx)
                    : OP == MM_DW ? mm_rsrc(x + (size_t)(t.row0 + s * ZS) * ldx, zleft * ldx)
                                  : rp;
#pragma unroll
    for (int i = 0; i < CQ; i++) {
      lds_void *dst = (lds_void *)(lq + i * NW * 1024);
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
        const uint32_t v = vp - cp + c + (uint32_t)(i * DP) * ldx;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sp, dst, 16, (int)(TP_T || (int)c < left ? v : kOutside),
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
#pragma unroll
      for (int j = 0; j < NQ; j++)
#pragma unroll
        for (int i = 0; i < NP; i++) acc[i][j] = M::mma(fp[h][i], fq[h][j], acc[i][j]);
    };
    read(0);
    if (GATHER) {
      mul(0);
      __builtin_amdgcn_sched_barrier(0);
    }
    read(1);
    if (s + 1 < steps) {
      wait_lgkm0();                      // the stage is free once every wave has read it
      mm_barrier();
      load(s + 1);
      gather_rows(s + 2);
    }
    if (!GATHER) mul(0);
    mul(1);
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
  mm_by_output(a.splits > 1 ? MM_PART : a.out_type, [&](auto out) {
    constexpr int OUT = decltype(out)::value;
    constexpr bool WIDE = OUT == MM_FP32 || OUT == MM_PART, NT = OP == MM_DW && OUT != MM_PART;
    constexpr int RB = WIDE ? 64 * 4 + 16 : 64 * 2 + 16;   // a row, and 16 bytes that spread the rows over the banks
    constexpr int LR = WIDE ? 16 : 8, CW = 64 / LR;        // lanes a row, columns a lane
    const long outs = OP == MM_DW ? (long)a.E * a.N : (long)a.R;
    float *part = a.part + (OUT == MM_PART ? (long)blockIdx.y * outs * pn : 0);
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
          if constexpr (OUT == MM_PART) *(v4i *)(part + at) = d;
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
  mm_by_output(a.out_type, [&](auto out) {
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

template <int OP, int TYPE, int BQ, int BP, int WQ, int WP, int MINW>
static hipError_t launch_tile(const MmArgs &a, hipStream_t s) {
  const long pn = OP == MM_FORWARD ? a.N : a.K, ptiles = (pn + BP - 1) / BP;
  long blocks;
  if (OP == MM_DW) blocks = 8l * a.E * (((a.N + BQ - 1) / BQ * ptiles + 7) / 8);
  else blocks = (((a.R + BQ - 1) / BQ + (a.first ? (a.E < a.R ? a.E : a.R) : 0)) * ptiles + 7) / 8 * 8;
  if (blocks > INT32_MAX / (64 * WQ * WP)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks, (unsigned)a.splits), threads(64 * WQ * WP);
  if (OP != MM_DX && a.rows) hipLaunchKernelGGL((k_mm_tile<OP, TYPE, BQ, BP, WQ, WP, true, MINW>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((k_mm_tile<OP, TYPE, BQ, BP, WQ, WP, false, MINW>), grid, threads, 0, s, a);
  if (a.splits > 1) {
    const long outs = OP == MM_DW ? (long)a.E * a.N : (long)a.R;
    hipLaunchKernelGGL(k_mm_join<TYPE>, dim3((unsigned)outs), dim3(256), 0, s, a);
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

template <int TYPE, bool GATHER>
__global__ __launch_bounds__(64 * kStreamWaves) void k_mm_stream(MmArgs a) {
  typedef MmElem<TYPE> M;
  typedef typename M::acc Acc;
  constexpr int ES = sizeof(typename M::t), D = kStreamSlots, NW = kStreamWaves;
  constexpr int kSlot = 4096;            // 16 weight rows, 16 rows of x
  constexpr int RS = 16 + 4;             // a row of sums, padded so that rows start on other banks
  __shared__ __align__(1024) uint8_t ring[NW][D][kSlot];
  __shared__ Acc sum[NW * 16 * RS / 4];
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  MmTile t;
  if (!mm_find_tile<16>(a, (a.N + 15) >> 4, t)) return;
  const int p0 = t.pt * 16, l16 = lane & 15, g = lane >> 4;
  const uint32_t ld = (uint32_t)a.K * ES;
  const int units = (int)((ld + 127) >> 7);
  const Rsrc wb = mm_rsrc((const uint8_t *)a.w + ((size_t)t.e * a.N + p0) * ld, (uint32_t)min(16, a.N - p0) * ld);
  // loads: row 8 i + lane / 8, its chunk swizzled as in the tile kernels
  uint32_t vw[2], ck[2];
  const uint8_t *xp[2];
  bool live[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int r = 8 * i + (lane >> 3);
    ck[i] = (uint32_t)((lane & 7) ^ swz_r(r)) * 16;
    vw[i] = (uint32_t)r * ld + ck[i];
    const long xr = r < t.rows ? (GATHER ? mm_x_row(a, t.row0 + r) : (long)t.row0 + r) : -1;
    live[i] = xr >= 0;
    xp[i] = (const uint8_t *)a.x + (live[i] ? (size_t)xr * ld : 0) + ck[i];
  }
  // this thread's outputs after the join: four channels of one row, and their scales
  const int oq = threadIdx.x >> 2, op = (threadIdx.x & 3) * 4;
  const bool writes = oq < t.rows && p0 + op < a.N;
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

  // XI: loads of eight rows of x a column
  auto body = [&](auto xi) {
    constexpr int XI = decltype(xi)::value, CNT = 2 + XI;
    auto load = [&](int s) {
      const uint32_t k = (uint32_t)(s * NW + w) * 128;
      uint8_t *dst = &ring[w][s % D][0];
#pragma unroll
      for (int i = 0; i < 2; i++)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wb, (lds_void *)(dst + i * 1024), 16,
                                                 (int)(k + ck[i] < ld ? vw[i] : kOutside), (int)k, 0, 0);
#pragma unroll
      for (int i = 0; i < XI; i++) {
        const uint8_t *p = live[i] && k + ck[i] < ld ? xp[i] + k : (const uint8_t *)g_mm_zeros;
        __builtin_amdgcn_global_load_lds(p, (lds_void *)(dst + 2048 + i * 1024), 16, 0, 0);
      }
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
      stream_read(rd0 + o, rd1 + o, rd0 + o + 2048, rd1 + o + 2048, fw, fx);
      acc = M::mma(fw[0], fx[0], acc);
      acc = M::mma(fw[1], fx[1], acc);
    }
  };
  // rows past XI * 8 of x are not loaded: their MFMA columns hold what LDS held and are not stored
  if (t.rows <= 8) body(MmConst<1>{});
  else body(MmConst<2>{});
  // sums of the waves: [wave][row][channel]
  sum[((w * 16 + l16) * RS + 4 * g) >> 2] = acc;
  __syncthreads();
  mm_by_output(a.out_type, [&](auto out) {
    constexpr int OUT = decltype(out)::value;
    if (!writes) return;
    Acc r = sum[(oq * RS + op) >> 2];
#pragma unroll
    for (int v = 1; v < NW; v++) r += sum[((v * 16 + oq) * RS + op) >> 2];
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      if constexpr (TYPE == MM_I8) v[k] = mm_scaled(r[k], mm_scale(xs), mm_scale(ws[k]));
      else v[k] = r[k];
    }
    mm_store4<OUT>(a, (long)(t.row0 + oq) * a.N + p0 + op, v);
  });
}

template <int TYPE>
static hipError_t launch_stream(const MmArgs &a, hipStream_t s) {
  const long tiles = (a.R + 15) / 16 + (a.first ? (a.E < a.R ? a.E : a.R) : 0);
  const long blocks = (tiles * ((a.N + 15) / 16) + 7) / 8 * 8;
  if (a.rows) hipLaunchKernelGGL((k_mm_stream<TYPE, true>), dim3((unsigned)blocks), dim3(64 * kStreamWaves), 0, s, a);
  else hipLaunchKernelGGL((k_mm_stream<TYPE, false>), dim3((unsigned)blocks), dim3(64 * kStreamWaves), 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------ the choice
//
// Tile shapes, all of four waves, and the blocks of each that a CU holds; weight:
// what covering an output element costs beside 256 x 128 once the chip is full
// (16384 x 4096 x 4096, over one and 32 groups: 435, 432, 481, 616 us and 517, 494,
// 572, 697 us).
enum { kShapes = 4 };
static const struct { int bq, bp, occ; float weight; } kMmShapes[kShapes] = {
    {256, 128, 2, 1.0f}, {128, 256, 2, 1.04f}, {128, 128, 3, 1.2f}, {64, 128, 4, 1.5f}};

MmPlan mm_plan(int op, int type, long E, long R, long N, long K) {
  MmPlan m = {0, 0, 1, 16, 16, 0};
  const long item = type == MM_I8 ? 1 : 2, groups = E < R ? E : R;
  const long pn = op == MM_FORWARD ? N : K, qn = op == MM_DW ? N : R, outs = op == MM_DW ? E * N : R;
  // Few rows a group: the weights pass once, 16 of their rows a block.  Short rows
  // make for blocks that mostly start and end (64 groups of 5 rows, N = 1024:
  // K = 512 in 21.0 us, in tiles 16.2; K = 2048 in 53.0, in tiles 58.4), which
  // costs nothing while tiles would leave most of the chip idle (64 groups of 8,
  // N = 256, K = 512: 6.4, 8.5 us).  Up to there more rows stream too, though
  // every 16 read the weights again (R = 64, N = 2048, K = 7168: 13.3, 17.6 us;
  // R = 128, N = 512, K = 2048: 5.8, 12.3; 8 groups of 24, N = 2048, K = 7168:
  // 68.2, 54.7).
  if (op == MM_FORWARD) {
    const long tiles16 = ((R + 15) / 16 + (E > 1 ? groups : 0)) * ((N + 15) / 16);
    const bool few = (R <= 8 * E || R <= 16) && K * item >= 4096 && tiles16 < 1l << 23;
    if (few || (R <= 64 * E && tiles16 <= 2048) || (R <= 128 && tiles16 <= 1024)) {
      m.stream = 1;
      return m;
    }
  }
  // The shape whose full rounds of blocks cover the least output.  Row tiles are
  // estimated for groups of even size, half a tile a group lost.
  long tiles = 0;
  float least = 0.f;
  for (int i = 0; i < kShapes; i++) {
    const auto &s = kMmShapes[i];
    if (op == MM_DW && i != 0 && i != 2) continue;
    long rows = (qn + s.bq - 1) / s.bq;
    if (op == MM_DW) rows *= E;
    else if (E > 1) rows = (R + groups * (s.bq / 2)) / s.bq > groups ? (R + groups * (s.bq / 2)) / s.bq : groups;
    const long n = rows * ((pn + s.bp - 1) / s.bp), slots = 256l * s.occ;
    const float cost = (float)((n + slots - 1) / slots * s.occ) * (float)(s.bq * s.bp) * s.weight;
    if (!tiles || cost < least) m.shape = i, least = cost, tiles = n;
  }
  // Short weight gradients write more than they read, and more blocks store better
  // (64 groups of 32 rows, 576 x 7168: 105 us, 118 in 256 x 128; 16 groups of 256,
  // 2048 x 2048: 45, 50; but 32 groups of 512, 1024 x 6144: 282, 251).
  if (op == MM_DW && R <= 256 * E) m.shape = 2;
  // Too few tiles for the chip: the reduction is split into as many parts as take
  // least time.  The estimate is fitted to whole and split times: a step takes 0.6 us
  // (1 us with transposed reads of both operands), all blocks' steps no less than
  // their loads at 12 TB/s (not a bound: full rounds of blocks fill LDS at 14 to 16);
  // the second launch, which joins the parts in order, 4 us, and their bytes twice at
  // 4 TB/s (R = 256, N = 1024, K = 4096: 15.2 us, 41.3 us whole; int8, R = 500,
  // N = 4608, K = 7168: 45.4 us in parts that fill the chip, 39.6 whole).
  const auto &shape = kMmShapes[m.shape];
  m.rows = shape.bq, m.cols = shape.bp;
  const long steps = op == MM_FORWARD ? K * item / 128 : op == MM_DX ? N / 64 : R / E / 64;
  const float step = op == MM_DW ? 1.0f : 0.6f;
  const float feed = (float)(tiles * steps * (shape.bq + shape.bp)) * (128 / 12e6f);
  float best = steps * step > feed ? steps * step : feed;
  for (long n = 2; n <= 16 && n * tiles <= 256l * shape.occ; n++) {
    const float run = (float)((steps + n - 1) / n) * step;
    const float us = (run > feed ? run : feed) + 4.0f + (float)(n * outs * pn) * 2e-6f;
    if (us < best) best = us, m.splits = (int)n;
  }
  if (m.splits > 1) m.scratch = (size_t)m.splits * outs * pn * 4;
  return m;
}

template <int OP, int TYPE>
static hipError_t launch_rows(const MmArgs &a, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_tile<OP, TYPE, 256, 128, 2, 2, 2>(a, s);
    case 1: return launch_tile<OP, TYPE, 128, 256, 2, 2, 2>(a, s);
    case 2: return launch_tile<OP, TYPE, 128, 128, 2, 2, 3>(a, s);
    default: return launch_tile<OP, TYPE, 64, 128, 2, 2, 4>(a, s);
  }
}

template <int TYPE>
static hipError_t launch_forward(const MmArgs &a, const MmPlan &m, hipStream_t s) {
  return m.stream ? launch_stream<TYPE>(a, s) : launch_rows<MM_FORWARD, TYPE>(a, m.shape, s);
}

template <int TYPE>
static hipError_t launch_16bit(const MmArgs &a, const MmPlan &m, hipStream_t s) {
  if (a.op == MM_FORWARD) return launch_forward<TYPE>(a, m, s);
  if (a.op == MM_DX) return launch_rows<MM_DX, TYPE>(a, m.shape, s);
  return m.shape == 2 ? launch_tile<MM_DW, TYPE, 128, 128, 2, 2, 3>(a, s) : launch_tile<MM_DW, TYPE, 256, 128, 2, 2, 2>(a, s);
}

hipError_t launch_mm(const MmArgs &args, hipStream_t s) {
  const MmPlan m = mm_plan(args.op, args.type, args.E, args.R, args.N, args.K);
  MmArgs a = args;
  a.splits = m.splits;
  return a.type == MM_I8     ? launch_forward<MM_I8>(a, m, s)
         : a.type == MM_BF16 ? launch_16bit<MM_BF16>(a, m, s)
                             : launch_16bit<MM_FP16>(a, m, s);
}

}  // namespace moe
