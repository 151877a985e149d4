// Ragged expert products for gfx950: forward, row gradient and weight gradient
// over 16-bit operands, the forward product over 8-bit integers, and the choice of
// shapes for these and the products built on them.
#include "moe_mm_tile.h"

namespace moe {

// ------------------------------------------------------------ the choice
//
// Tile shapes, all of four waves, and the blocks of each that a CU holds; weight:
// what covering an output element costs beside 256 x 128 once the chip is full
// (16384 x 4096 x 4096, over one and 32 groups: 435, 432, 481, 616 us and 517, 494,
// 572, 697 us).
enum { kShapes = 4 };
static const struct { int bq, bp, occ; float weight; } kMmShapes[kShapes] = {
    {256, 128, 2, 1.0f}, {128, 256, 2, 1.04f}, {128, 128, 3, 1.2f}, {64, 128, 4, 1.5f}};
// 8-bit floating point, by fp16 instructions: one group of that size 537, 497, 550, 586 us,
// and with every lane's conversions in front of the products a tile that has its SIMDs to
// itself pays for its size (20 groups of 30 rows on average, 2040 x 6816: 266, 252, 128, 88
// us): kF8xFew of launches of up to kF8xFewTiles tiles.  Over 14 drawn calls that this was
// not fitted to, the choice took at most 3 % longer than the best shape.
static const int kF8xOcc[kShapes] = {2, 2, 2, 4};
static const float kF8xWeights[kShapes] = {0.98f, 0.95f, 1.02f, 1.08f}, kF8xFew[kShapes] = {1.3f, 1.3f, 1.2f, 1.0f};
static const int kF8xFewTiles[kShapes] = {384, 384, 512, 0};
// By the 8-bit instruction: 313, 295, 312, 356 us; 64-row tiles read the weights of more
// groups twice (384 groups of 64 rows on average, 1152 x 7168: 891, 630, 681, 734 us) and
// weigh as the mean over 28 timed calls has it (2.7 % more than the best shape, 21 % in the
// worst).
static const float kF8Weights[kShapes] = {1.0f, 0.95f, 1.05f, 1.35f};

// Steps that a tile's start and end cost, fitted to 50 drawn sizes: in the gated block
// little more than a product's, whose rounds are compared by their steps alone; with the
// activation's gradient, which moves 10 bytes an output, what smaller tiles have less of
// (6546 rows, 240 x 2040: 48.3 us in 128 x 256, 29.8 in 64 x 128).
static const float kGluStart[kShapes] = {9.f, 8.f, 7.f, 6.f}, kGradStart[kShapes] = {40.f, 38.f, 25.f, 17.f};

// built: a product that mm_tail and the starts above are for (op as the product's).
enum { kPlain = 0, kBuilt = 1, kBuiltGrad = 2 };
static MmPlan shape_plan(int op, int type, long E, long R, long N, long K, int built) {
  MmPlan m = {0, 0, 1, 16, 16, 0, 0};
  const long item = type == MM_I8 || type == MM_F8 || type == MM_F8X ? 1 : 2, groups = E < R ? E : R;
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
  const long steps = op == MM_FORWARD ? K * item / 128 : op == MM_DX ? N / 64 : R / E / 64;
  auto start = [&](int i) {
    return !built ? 0.f : built == kBuiltGrad ? kGradStart[i] : type == MM_F8X ? 0.5f * kGluStart[i] : kGluStart[i];
  };
  auto occ = [&](int i) { return type == MM_F8X ? kF8xOcc[i] : kMmShapes[i].occ; };
  auto weight = [&](int i) { return type == MM_F8X ? kF8xWeights[i] : type == MM_F8 ? kF8Weights[i] : kMmShapes[i].weight; };
  for (int i = 0; i < kShapes; i++) {
    const auto &s = kMmShapes[i];
    if (op == MM_DW && i != 0 && i != 2) continue;
    long rows = (qn + s.bq - 1) / s.bq;
    if (op == MM_DW) rows *= E;
    else if (E > 1) rows = (R + groups * (s.bq / 2)) / s.bq > groups ? (R + groups * (s.bq / 2)) / s.bq : groups;
    const long n = rows * ((pn + s.bp - 1) / s.bp), slots = 256l * occ(i);
    float cost = (float)((n + slots - 1) / slots * occ(i)) * (float)(s.bq * s.bp) * weight(i);
    if (built) cost *= (float)steps + start(i);
    if (type == MM_F8X && n <= kF8xFewTiles[i]) cost *= kF8xFew[i];
    if (!tiles || cost < least) m.shape = i, least = cost, tiles = n;
  }
  // Short weight gradients write more than they read, and more blocks store better
  // (64 groups of 32 rows, 576 x 7168: 105 us, 118 in 256 x 128; 16 groups of 256,
  // 2048 x 2048: 45, 50; but 32 groups of 512, 1024 x 6144: 282, 251).
  if (op == MM_DW && R <= 256 * E) m.shape = 2;
  // Too few tiles for the chip: the reduction is split into as many parts as take
  // least time.  The estimate is fitted to whole and split times: a step takes 0.6 us
  // (1 us with transposed reads of both operands and with conversions, 0.8 by the 8-bit
  // floating-point instruction), all blocks' steps no less than
  // their loads at 12 TB/s (not a bound: full rounds of blocks fill LDS at 14 to 16);
  // the second launch, which joins the parts in order, 4 us, and their bytes twice at
  // 4 TB/s (R = 256, N = 1024, K = 4096: 15.2 us, 41.3 us whole; int8, R = 500,
  // N = 4608, K = 7168: 45.4 us in parts that fill the chip, 39.6 whole).
  const auto &shape = kMmShapes[m.shape];
  m.rows = shape.bq, m.cols = shape.bp;
  const float step = op == MM_DW || type == MM_F8X ? 1.0f : type == MM_F8 ? 0.8f : 0.6f;
  const float feed = (float)(tiles * steps * (shape.bq + shape.bp)) * (128 / 12e6f);
  float best = steps * step > feed ? steps * step : feed;
  for (long n = 2; n <= 16 && n * tiles <= 256l * occ(m.shape); n++) {
    const float run = (float)((steps + n - 1) / n) * step;
    const float us = (run > feed ? run : feed) + 4.0f + (float)(n * outs * pn) * 2e-6f;
    if (us < best) best = us, m.splits = (int)n;
  }
  if (m.splits > 1) m.scratch = (size_t)m.splits * outs * pn * 4;
  if (!built || m.splits > 1) return m;
  // The last round in parts (mm_tail), in the shapes of two blocks a CU, where its share
  // of a round and the second launch (about 12 us for a round's parts, in rounds of 1.5 us
  // a step) cost less than what the best whole rounds do: 32 groups of 512 rows on average
  // with loads of rank^-0.5, row gradient 1024 x 6144 to the projections 323 -> 267 us; 4097
  // rows, 2 x 2304 x 7168 242 -> 233 us.  Launches of less than a round gain where the
  // reduction is long (64 groups of 2 rows on average, 576 x 7168, row gradient: 110 -> 77
  // us) and lose where it is short (190 rows, 2 x 2024 x 1280: 11.1, 23.0 us; 1302 rows,
  // 8 bits, 2 x 2152 x 2544: 44.7, 57.4).
  for (int i = 0; i < 2; i++) {
    const auto &s = kMmShapes[i];
    const long rows = E > 1 ? ((R + groups * (s.bq / 2)) / s.bq > groups ? (R + groups * (s.bq / 2)) / s.bq : groups)
                            : (R + s.bq - 1) / s.bq;
    const long slots = 256l * occ(i), n = rows * ((pn + s.bp - 1) / s.bp);
    if (n > 1l << 23) continue;
    const MmTail t = mm_tail((int)n, (int)slots, (int)steps);
    if (t.parts < 2 || (t.full == 0 && steps < 64)) continue;
    const float cost = ((float)(t.full / slots) * ((float)steps + start(i)) + (1.0f / t.parts + 0.05f) * (float)steps + 8.0f) *
                       occ(i) * (float)(s.bq * s.bp) * weight(i);
    if (cost < least) least = cost, m.shape = i, m.tail = 1, m.rows = s.bq, m.cols = s.bp;
  }
  if (m.tail) m.scratch = 256l * occ(m.shape) * kMmShapes[m.shape].bq * kMmShapes[m.shape].bp * 4;
  return m;
}

// A gated block is chosen for as the product with both its branches' channels.
MmPlan mm_plan(int op, int type, long E, long R, long N, long K) {
  if (op == MM_GLU_DX) return shape_plan(MM_DX, type, E, R, N, K, kBuiltGrad);
  if (op != MM_GLU) return shape_plan(op, type, E, R, N, K, type == MM_F8 || type == MM_F8X ? kBuilt : kPlain);
  MmPlan m = shape_plan(MM_FORWARD, type, E, R, 2 * N, K, kBuilt);
  m.cols /= 2;
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
  return m.stream ? launch_stream<MM_FORWARD, TYPE>(a, s) : launch_rows<MM_FORWARD, TYPE>(a, m.shape, s);
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
  a.splits = m.splits, a.tail = m.tail;
  if (a.type == MM_F8 || a.type == MM_F8X) return launch_fp8(a, m, s);
  if (a.op == MM_GLU || a.op == MM_GLU_DX) return launch_glu(a, m, s);
  return a.type == MM_I8     ? launch_forward<MM_I8>(a, m, s)
         : a.type == MM_BF16 ? launch_16bit<MM_BF16>(a, m, s)
                             : launch_16bit<MM_FP16>(a, m, s);
}

}  // namespace moe
