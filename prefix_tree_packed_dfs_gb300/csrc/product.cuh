// The matrix products of the projections and the feed-forward block, with
// their epilogues (linear.cu, ffn.cu).  A product is  D[m, n] = sum_k A B  over
// bf16 operands, fp32 sums:
//   kLin      x w^T              act(z + bias) + residual
//   kDz       x w^T              dz = dy act'(z + bias), its column sums
//   kDx       dz w               stored
//   kDw       dz^T x             stored
//   kGate     x (w_gate | w_up)^T   a = act(g) u (and g, u kept)
//   kGateBwd  dy w_out              dg = da u act'(g), du = da act(g)
//   kGrads    the kDx and kDw products of a small backward in one launch
// The tiles that are left over from whole rounds of kLin, kDx and kDw may be
// split over K (split_of): fp32 partial tiles, summed in a fixed order by
// linear.cu's join_kernel, which then does the epilogue.
//
// 256 x 256 tiles on a pair of CTAs (tcgen05 cta_group::2): each CTA holds 128
// rows of A, 128 of B and its 128 rows of the result.  64 elements of K per
// stage, the stages filled by TMA; two accumulators of 256 TMEM columns, so that
// a tile's epilogue runs under the next tile's products.  Results leave through
// shared memory by TMA; what an epilogue reads besides (residual, dy, g and u)
// comes in by TMA to the very places its results leave from, issued when the tile
// before has left and so long before the accumulator is ready.  kDx, kDw and kGate
// read nothing, let a warpgroup's results leave through one box and have six
// stages (tensor pipe 88-90% of the cycles); the others have five and two boxes.
// (Residual, dy, g and u by plain loads of 64 bytes per row and thread, one chunk
// ahead and with L2 prefetches, six stages for all: kDz 188 us against 169,
// kGateBwd 250 against 189 at 8,192 rows.)
// kGate takes 128 rows of the gate's weights and 128 of the up projection's as
// one B tile (one of each per CTA), so a thread's accumulator row holds g and u
// of the same channels.
// kGateBwd moves 64 columns of g and u in and of dg and du out at a time, through
// two places; warp 3 carries them, so that a place is filled again, for the next
// tile too, as soon as its results have left.  Its g and u come in beside operands
// that take 64 bytes per cycle and SM alone: 32,768 rows, widths 2,048 and 8,192,
// 711 us (1.55 PFLOP/s) against 545 for the same product without them.  (Four
// stages and three places 790 us, boxes of 32 columns 740, g and u sent ahead to
// L2 776.)
// The tensor core adds to its fp32 accumulator with truncation: 1e-7 of the
// running sum per step of 16 elements of K.  The sums over rows (kDw) and over
// the wide side (kDx) stop every 8,192 elements and are added up in registers
// with rounding to nearest: at most 5e-5 is left, a fortieth of the results'
// bf16 rounding; sums over at most kMostK channels (2e-4 at most) need no stop.
// g and u are kept for the backward in 16 bits: as fp16 scaled by a power of two
// for every 32 channels of a row, so that the largest lies in [2^14, 2^15).  That
// is eight times as precise as bf16 for the same bytes, at any scale (a value
// 2^-29 of its group's largest still has its 11 bits); with g and u in bf16 the
// gradients' error over fp64 was 3.0e-3 of their norm against 2.4e-3 with them
// unrounded, of which 1.7e-3 is the results' own rounding.
// A few tiles leave most SMs idle and wait for their epilogue at the end: kLin, kDz,
// kDx and kDw then take tiles half as wide (256 x 128, plan_of), and up to four pairs
// of a cluster share a tile's K: each leaves its sums in shared memory, where the
// stages were, and takes a part of the rows out, adding the pairs' sums up in their
// order through distributed shared memory (a warp reads whole rows: 16 bytes of 32
// rows each took 4 us longer).  (1,003 rows, widths 5,456 to 1,000:
// 17 us against 28 in narrow tiles alone; 256 rows, 8,192 to 256: 12 against 16.)
// A small backward's products that do not wait for one another (dx, dw; the block's
// dx, dw_in, dw_out) are one launch of narrow tiles, the longest sums first (kGrads,
// grads_plan); a pair that has one of those takes fewer of the others.  (1,003 rows
// back through 1,000 -> 2,728 -> 1,000: 34 us against 51 in three.)
// Kernels of one call overlap (programmatic dependent launch): each sets itself
// up under the one before and then waits for it.  A product that needs nothing of
// the one before, where that one leaves SMs free (early), takes them at once and
// waits at its end, so that a kernel that is done means that those before it are
// (1,001 rows, widths 1,000 and 552, forward and backward: 50 us against 56; beside
// a product that fills the GPU it costs 1%).
// Warps of a CTA: 0 TMA producer, 1 MMA issuer (of the pair's first CTA), 2
// TMEM owner, 3 kGateBwd's carrier, 4-11 epilogue (two warpgroups).  CTAs are
// persistent and walk the tiles in panels of 8 columns of tiles, so that the pairs
// running together share rows of A and of B in L2.
// What bounds it: the tensor pipe, then the power limit (8,192 rows: gate 2 x
// 2,048 x 8,192 294 us, 1.87 PFLOP/s; dx 285, dw 275; 96,888 rows of 2,048 onto the
// residual stream 442 us, 1.84 PFLOP/s; long runs settle at 1.6-1.7).
#pragma once
#include <type_traits>

#include "activation.cuh"
#include "pair.cuh"
#include "rowwise.cuh"

namespace tpk {
namespace product {

constexpr int kTile = 256;             // rows (and, but for kGate, columns) of a pair's tile
constexpr int kHalf = 128;             // rows of A / of B a CTA holds
constexpr int kBoxBytes = kHalf * 128; // 128 rows of 64 bf16
constexpr int kThreads = 384;
constexpr int kEpiThreads = 256;
constexpr int kPanel = 8;
constexpr int kChunk = 128;            // stages per accumulation of kDx, kDw
constexpr int kMostK = 32768;          // channels of a sum that never stops
constexpr int kPairs = 76;             // pairs a split over K aims to fill
constexpr int kTeams = 4;              // pairs of a cluster at most
constexpr int kClusters4 = 36, kClusters8 = 15;   // clusters of 4 and 8 CTAs that 152 SMs hold at once, one CTA each
constexpr int kGroup = 32;             // channels that share a power of two in what kGate keeps
// The chunked epilogue holds 128 columns of a row per thread: the other warps
// give registers to its two warpgroups.
constexpr uint32_t kRegsCtl = 56;
constexpr uint32_t kRegsEpi = 216;
constexpr int kRegsNeeded = 128 * kRegsCtl + 256 * kRegsEpi;

enum Mode { kLin = 0, kDz = 1, kDx = 2, kDw = 3, kGate = 4, kGateBwd = 5, kGrads = 6 };

struct Maps {
  CUtensorMap a, b, b2;      // b2: kGate's up rows
  CUtensorMap in, in2;       // kLin residual, kDz dy; kGateBwd g, u
  CUtensorMap out, out2, out3;   // kGate: a, g, u; kGateBwd: dg, du
  CUtensorMap more;
  // kGrads: of the s-th product
  __host__ __device__ const CUtensorMap& grad_a(int s) const { return s == 0 ? a : s == 1 ? in : more; }
  __host__ __device__ const CUtensorMap& grad_b(int s) const { return s == 0 ? b : s == 1 ? b2 : in2; }
  __host__ __device__ const CUtensorMap& grad_out(int s) const { return s == 0 ? out : s == 1 ? out2 : out3; }
};

// One of kGrads' products.
struct Sub {
  int32_t M, N, k_iters;
  int32_t amn;               // A stored with M contiguous (dw)
  int32_t mt, nt;
};

struct Params {
  int32_t M, N, K;           // extents of the product (kGate, kGateBwd: N = channels of one of the two)
  int32_t whole, splits;     // tiles before the split ones; splits of each of those (split_of)
  int32_t act;
  int32_t has_in;            // kLin: a residual
  const uint16_t* in;        // teams: residual or dy, and the result, which leave their rows' maps unused
  uint16_t* out;
  int64_t ld_in, ld_out;
  int32_t save;              // kGate: g and u go out too
  int32_t early;             // needs nothing of the kernel before, only of those that it waited for
  int32_t narrow;            // tiles of 128 columns (the kernel knows by its type)
  int32_t teams;             // pairs that share a tile's K (the kernel knows by its cluster); > 1: one tile each
  int32_t late;              // lets the next kernel start only after its own wait (that one may be early)
  const float* bias;         // [N] or nullptr
  float* colsum;             // kDz: [ceil(M / 32)][N] sums of 32 rows of dz; nullptr: none
  float* acc;                // splits > 1: [splits][tiles - whole][256 * 256]
  uint8_t* exps;             // kGate, kGateBwd: [2][groups][exp_rows] biased exponents of g's and u's largest
  int64_t exp_rows;
  Sub sub[3];                // kGrads, by falling k_iters
  int32_t* err;
};

template <int kMode>
struct Smem {
  static constexpr bool kSix = kMode == kDx || kMode == kDw || kMode == kGate || kMode == kGrads;
  static constexpr int kStages = kSix ? 6 : 5;
  static constexpr int kBoxes = kSix ? 1 : 2;
  uint8_t a[kStages][kBoxBytes];
  uint8_t b[kStages][kBoxBytes];
  uint8_t out[2][kBoxes][kBoxBytes];        // two boxes per warpgroup; kGateBwd: two places of g and u
  float bias[2][kHalf];                // of the tile at hand, per warpgroup
  uint64_t full[kStages], empty[kStages];
  uint64_t tm_full[2], tm_empty[2];
  uint64_t in_full[2][2], written[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  uint32_t issued;   // stages the producer has filled
};
template <int kMode>
constexpr size_t kSmemBytes = sizeof(Smem<kMode>) + 1024;
static_assert(kSmemBytes<kLin> <= 227 * 1024 && kSmemBytes<kDx> <= 227 * 1024, "shared memory");

// The split over K.  Pairs take tiles in rounds; the `tail` tiles left over from
// whole rounds (all of them, if they are few) take a round of their own, which
// `splits` units for each of them make shorter.  It has to pay for the partial
// tiles (written and read once, at about 5 TB/s) and for the joining kernel.
struct Split {
  int64_t whole, tail;
  int splits;
};
// us: of the last round.
inline Split split_of(int64_t tiles, int64_t k_iters, double* us_out = nullptr, bool may_split = true) {
  Split s{tiles, 0, 1};
  const int64_t tail = tiles % kPairs;
  const double tile_us = 0.27 * static_cast<double>(k_iters);   // 64 elements of K: 512 cycles
  double best = tile_us;
  if (us_out) *us_out = tail == 0 ? 0.0 : best;
  if (tail == 0 || !may_split) return s;
  for (int64_t n = 2; n <= k_iters / 4 && n <= (tail * 8 < kPairs ? kPairs / tail : 8); ++n) {
    const int64_t rounds = (tail * n + kPairs - 1) / kPairs;
    const double us = tile_us * static_cast<double>(rounds) / static_cast<double>(n) + 6.0 +
                      0.105 * static_cast<double>(tail * n) + 0.1 * static_cast<double>(n);
    if (us < best) {
      best = us;
      s = Split{tiles - tail, tail, static_cast<int>(n)};
    }
  }
  if (us_out) *us_out = best;
  return s;
}

// How a product is done: in wide tiles, some of them split, or in narrow ones.
// Those need 256 cycles for 64 elements of K where few pairs run, about 384 where
// the operands' way into the SMs is full, and half of the 2.2 us that a lone wide
// tile's epilogue takes; where few columns are left of the last wide tile they are
// quicker in any number.  (1,000 rows, widths 1,000 and 552, gelu: 10.7 us in narrow
// tiles, 14.5 in wide ones; 200 rows, widths 1,024 and 256: 7.2 against 10.5.)  A team
// of pairs divides the stages and pays about 2.2 us to meet.
struct Plan {
  bool narrow;
  int teams;
  Split split;
  double us;     // estimate, without the kernel's start and end
};
inline Plan plan_of(int64_t M, int64_t N, int64_t K, bool may_split = true) {
  const int64_t mt = (M + kTile - 1) / kTile, wide = mt * ((N + kTile - 1) / kTile);
  const int64_t narrow = mt * ((N + kHalf - 1) / kHalf), k_iters = (K + 63) / 64;
  double us;
  Plan p{false, 1, split_of(wide, k_iters, &us, may_split), 0.0};
  p.us = us + 2.2 + 0.27 * static_cast<double>((p.split.tail ? p.split.whole : wide - wide % kPairs) / kPairs * k_iters);
  const int64_t rounds = (narrow + kPairs - 1) / kPairs;
  const double stage_us = narrow <= kPairs / 2 ? 0.14 : 0.2;
  const double alone = stage_us * static_cast<double>(rounds * k_iters) + 1.1;
  if (alone < p.us && k_iters <= kChunk) p = Plan{true, 1, Split{narrow, 0, 1}, alone};
  for (int teams = 2; teams <= kTeams; teams *= 2) {
    const int64_t each = (k_iters + teams - 1) / teams;
    if (narrow > (teams == 2 ? kClusters4 : kClusters8) || k_iters < 2 * teams || each > kChunk) continue;
    const double together = stage_us * static_cast<double>(each) + 1.1 + 2.2;
    if (together < p.us) p = Plan{true, teams, Split{narrow, 0, 1}, together};
  }
  return p;
}

// Unit u covers tile (m, n) and the stages [k0, k0 + nk) of K.
struct Shape {
  int mt, nt, units, k_iters;
};
struct Unit {
  int m, n, k0, nk;
  int split;                 // -1: the whole of K
  int tile;
  int sub;                   // kGrads
};
// Columns of a tile.
template <int kMode, bool kNarrow = false>
constexpr int kTileN = kMode == kGate || kNarrow ? kHalf : kTile;

template <int kMode, bool kNarrow = false>
__host__ __device__ inline Shape shape_of(const Params& p) {
  Shape s;
  s.mt = (p.M + kTile - 1) / kTile;
  s.nt = (p.N + kTileN<kMode, kNarrow> - 1) / kTileN<kMode, kNarrow>;
  s.k_iters = (p.K + 63) / 64;
  s.units = p.whole + (s.mt * s.nt - p.whole) * p.splits;
  return s;
}
// Tile t of the walk, in panels of kPanel columns of tiles.
__device__ __forceinline__ void place_of(int mt, int nt, int t, int& m, int& n) {
  const int panel = t / (kPanel * mt);
  t -= panel * kPanel * mt;
  const int width = min(kPanel, nt - panel * kPanel);
  m = t / width;
  n = panel * kPanel + t % width;
}
template <bool kNarrow>
__device__ __forceinline__ Unit unit_of(const Params& p, const Shape& s, int u, int team, int teams) {
  Unit w{0, 0, 0, s.k_iters, -1, 0, 0};
  if (kNarrow) {   // never split over units, but over the pairs of a cluster
    w.k0 = s.k_iters * team / teams;
    w.nk = s.k_iters * (team + 1) / teams - w.k0;
  } else if (u >= p.whole && p.splits > 1) {
    const int tail = s.mt * s.nt - p.whole;
    w.split = (u - p.whole) / tail;
    u = p.whole + (u - p.whole) % tail;
    w.k0 = static_cast<int>(static_cast<int64_t>(s.k_iters) * w.split / p.splits);
    w.nk = static_cast<int>(static_cast<int64_t>(s.k_iters) * (w.split + 1) / p.splits) - w.k0;
  }
  w.tile = u;
  place_of(s.mt, s.nt, u, w.m, w.n);
  return w;
}

// kGrads: the i-th tile of pair `pair` of `pairs`, if it has so many.  The first
// product's tiles go round; while some pairs do one more of those, the others do
// `e` of the shorter ones; the rest goes round.
__device__ __forceinline__ bool grad_unit(const Params& p, int pair, int pairs, int i, Unit& w) {
  const int n0 = p.sub[0].mt * p.sub[0].nt, n1 = p.sub[1].mt * p.sub[1].nt, n2 = p.sub[2].mt * p.sub[2].nt;
  const int extra = n0 % pairs, mine = n0 / pairs + (pair < extra ? 1 : 0);
  if (i < mine) {
    w.sub = 0;
    w.tile = pair + pairs * i;
  } else {
    i -= mine;
    const int rest = n1 + n2, idle = pairs - extra;
    const int e = extra > 0 ? p.sub[0].k_iters / p.sub[1].k_iters : 0;
    const int ahead = min(rest, idle * e);
    int v = -1;
    if (pair >= extra) {
      const int at = pair - extra, has = at < ahead ? (ahead - at - 1) / idle + 1 : 0;
      if (i < has) v = at + idle * i;
      i -= has;
    }
    if (v < 0) {
      v = ahead + pair + pairs * i;
      if (v >= rest) return false;
    }
    w.sub = v < n1 ? 1 : 2;
    w.tile = v < n1 ? v : v - n1;
  }
  const Sub& s = p.sub[w.sub];
  w.k0 = 0;
  w.nk = s.k_iters;
  w.split = -1;
  place_of(s.mt, s.nt, w.tile, w.m, w.n);
  return true;
}

__device__ __forceinline__ uint64_t pair_at(const uint32_t (&x)[32], int e) {
  return ptx::f2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
}

// 32 columns of a row into half `half` of a box of 64, in the TMA's 128-byte
// swizzle (16-byte piece i of row r at piece i ^ (r % 8)).
__device__ __forceinline__ void put64(uint8_t* box, int r, int half, const uint32_t (&o)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint4*>(box + r * 128 + (((half * 4 + q) ^ (r & 7)) * 16)) =
        make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
}
__device__ __forceinline__ void get64(const uint8_t* box, int r, int half, uint32_t (&o)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int4 v = ptx::lds128i(box + r * 128 + (((half * 4 + q) ^ (r & 7)) * 16));
    o[4 * q] = v.x; o[4 * q + 1] = v.y; o[4 * q + 2] = v.z; o[4 * q + 3] = v.w;
  }
}
// The biased exponent of the largest finite magnitude of x, within [15, 254].
__device__ __forceinline__ uint32_t largest_exponent(const uint32_t (&x)[32]) {
  float top[4] = {};
#pragma unroll
  for (int e = 0; e < 32; e += 2)
    top[(e / 2) & 3] = ptx::max3(top[(e / 2) & 3], fabsf(__uint_as_float(x[e])), fabsf(__uint_as_float(x[e + 1])));
  uint32_t m = __float_as_uint(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
  if (m >= 0x7f800000u) {   // an infinity has no say
    m = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint32_t v = x[e] & 0x7fffffffu;
      m = v < 0x7f800000u && v > m ? v : m;
    }
  }
  m >>= 23;
  return m < 15 ? 15 : m;
}
// The power of two that takes such a group to [2^14, 2^15), and its inverse.
__device__ __forceinline__ float group_scale(uint32_t e) { return __uint_as_float((268 - e) << 23); }
__device__ __forceinline__ float group_unscale(uint32_t e) { return __uint_as_float((e - 14) << 23); }

// Where the 16 bytes q of a row of 128 fp32 sums lie in a pair's shared memory.
__device__ __forceinline__ uint32_t team_place(int r, int q) {
  return static_cast<uint32_t>(r * 512 + ((q ^ (r & 31)) * 16));
}

// Sums over the warp's 32 rows of x[0..31] (a row per lane): lane l returns
// the sum of column l.  Each step halves the columns a lane holds.
__device__ __forceinline__ float column_sums(float (&x)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float send = up ? x[j] : x[j + o], keep = up ? x[j + o] : x[j];
      x[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return x[0];
}

// kOne: every tile is a single accumulation, which goes out while it is read
// from TMEM and need not be held whole.
template <int kMode, bool kOne, bool kNarrow>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  using Sm = Smem<kMode>;
  constexpr int kStages = Sm::kStages;
  Sm& S = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr bool kAmn = kMode == kDw;                                          // A stored with M contiguous
  constexpr bool kBmn = kMode == kDx || kMode == kDw || kMode == kGateBwd || kMode == kGrads;   // B with N contiguous
  constexpr bool kPlain = kMode == kLin || kMode == kDx || kMode == kDw || kMode == kGrads;
  static_assert(kOne || kMode == kDx || kMode == kDw, "sums over channels do not stop");
  static_assert(!kNarrow || (kOne && (kMode < kGate || kMode == kGrads)), "narrow tiles are whole sums");
  constexpr int kCols = kNarrow ? kHalf : kTile;   // columns of the accumulator
  constexpr int kBRows = kCols / 2;                // rows of B a CTA holds
  const int warp = threadIdx.x >> 5;
  const uint32_t place = ptx::cluster_rank(), size = ptx::cluster_size();
  const uint32_t rank = place & 1, lead = place & ~1u;         // of the pair, its first CTA
  const int team = static_cast<int>(place >> 1), teams = static_cast<int>(size >> 1);
  const int pair = static_cast<int>(blockIdx.x / size), n_pairs = static_cast<int>(gridDim.x / size);
  volatile int* abort_flag = &S.abort_flag;
  const Shape sh = shape_of<kMode, kNarrow>(p);
  auto next = [&](int i, Unit& w) {   // the pair's i-th unit
    if constexpr (kMode == kGrads) {
      return grad_unit(p, pair, n_pairs, i, w);
    } else {
      const int u = pair + i * n_pairs;
      if (u >= sh.units) return false;
      w = unit_of<kNarrow>(p, sh, u, team, teams);
      return true;
    }
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&S.full[s], 1);
      ptx::mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&S.tm_full[b], 1);
      ptx::mbar_init(&S.tm_empty[b], 2 * kEpiThreads / 32);   // every epilogue warp of the pair
      ptx::mbar_init(&S.in_full[0][b], 1);
      ptx::mbar_init(&S.in_full[1][b], 1);
      ptx::mbar_init(&S.written[b], kEpiThreads / 32);
    }
    ptx::mbar_init(&S.drain, 1);
    S.abort_flag = 0;
    S.issued = 0;
    ptx::fence_mbar_init();
  }
  __syncwarp();
  ptx::cluster_sync();   // the cluster's barriers exist
  if (!p.late) ptx::dependents_launch();
  if (!p.early) ptx::dependency_wait();   // what the kernel before wrote is there
  if (p.late) ptx::dependents_launch();
  // the producer needs no accumulator and is off
  uint32_t tmem = 0;
  if (warp == 2) {
    ptx::tmem_alloc_pair(&S.tmem_base, 2 * kCols);
    ptx::tmem_relinquish_pair();
    ptx::tc_fence_before();
  }
  if (warp > 0) {
    asm volatile("bar.sync 3, %0;" ::"n"(kThreads - 32) : "memory");
    ptx::tc_fence_after();
    tmem = S.tmem_base;
  }
  if (warp < 4) {
    if constexpr (!kOne) ptx::regs_dec<kRegsCtl>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (ptx::elect_one()) {
        ptx::prefetch_tensormap(&maps.a);
        ptx::prefetch_tensormap(&maps.b);
        const CUtensorMap* mb = kMode == kGate && rank == 1 ? &maps.b2 : &maps.b;
        uint32_t it = 0;
        bool ok = true;
        Unit w;
        for (int i = 0; ok && next(i, w); ++i) {
          const CUtensorMap* ma = kMode == kGrads ? &maps.grad_a(w.sub) : &maps.a;
          if (kMode == kGrads) mb = &maps.grad_b(w.sub);
          const bool amn = kMode == kGrads ? p.sub[w.sub].amn != 0 : kAmn;
          const int m0 = w.m * kTile + static_cast<int>(rank) * kHalf;
          const int n0 = w.n * kTileN<kMode, kNarrow> + (kMode == kGate ? 0 : static_cast<int>(rank) * kBRows);
          for (int k = 0; k < w.nk; ++k, ++it) {
            const int st = it % kStages;
            if (it >= kStages && !ptx::mbar_wait(&S.empty[st], (it / kStages - 1) & 1, abort_flag, kWaitLimitNs)) {
              ok = false;
              break;
            }
            if (rank == 0) ptx::mbar_arrive_expect_tx(&S.full[st], 2 * (kBoxBytes + kBRows * 128));
            const uint32_t bar = ptx::cluster_addr(&S.full[st], lead);
            const int kk = (w.k0 + k) * 64;
            if (amn) {
              ptx::tma_load_2d_pair(S.a[st], ma, bar, m0, kk);
              ptx::tma_load_2d_pair(S.a[st] + kBoxBytes / 2, ma, bar, m0 + 64, kk);
            } else {
              ptx::tma_load_2d_pair(S.a[st], ma, bar, kk, m0);
            }
            if constexpr (kBmn) {
              ptx::tma_load_2d_pair(S.b[st], mb, bar, n0, kk);
              if (kBRows > 64) ptx::tma_load_2d_pair(S.b[st] + kBoxBytes / 2, mb, bar, n0 + 64, kk);
            } else {
              ptx::tma_load_2d_pair(S.b[st], mb, bar, kk, n0);
            }
          }
        }
        S.issued = it;
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------------------------------------------------- MMA issuer
      if (ptx::elect_one()) {
        // K step of 16 elements: 32 bytes along a K-major row, 16 rows of 128
        // bytes of an MN-major box (its two 64-column boxes half a stage apart)
        constexpr uint32_t kStepB = kBmn ? 2048 : 32;
        uint32_t it = 0, tile = 0;
        bool ok = true;
        Unit w;
        for (int i = 0; ok && next(i, w); ++i) {
          const bool amn = kMode == kGrads ? p.sub[w.sub].amn != 0 : kAmn;
          const uint32_t step_a = amn ? 2048 : 32, lbo_a = amn ? kBoxBytes / 2 : 16;
          const uint32_t idesc =
              amn ? ptx::idesc_bf16_f32(kTile, kCols, true, kBmn) : ptx::idesc_bf16_f32(kTile, kCols, false, kBmn);
          const int per = kOne ? w.nk : kChunk;
          for (int k0 = 0; ok && k0 < w.nk; k0 += per, ++tile) {
            const uint32_t buf = tile & 1;
            if (tile >= 2 && !ptx::mbar_wait(&S.tm_empty[buf], (tile / 2 - 1) & 1, abort_flag, kWaitLimitNs)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const int nk = min(per, w.nk - k0);
            for (int k = 0; k < nk; ++k, ++it) {
              const int st = it % kStages;
              if (!ptx::mbar_wait(&S.full[st], (it / kStages) & 1, abort_flag, kWaitLimitNs)) {
                ok = false;
                break;
              }
              ptx::tc_fence_after();
              const uint64_t ad = ptx::sw128_desc(ptx::smem_addr(S.a[st]), lbo_a, 1024);
              const uint64_t bd = ptx::sw128_desc(ptx::smem_addr(S.b[st]), kBmn ? kBoxBytes / 2 : 16, 1024);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                ptx::mma_ss_pair(tmem + buf * kCols, ptx::desc_add(ad, q * step_a), ptx::desc_add(bd, q * kStepB),
                                 idesc, (k > 0 || q > 0) ? 1u : 0u);
              ptx::mma_commit_pair(&S.empty[st], lead);
            }
            if (ok) ptx::mma_commit_pair(&S.tm_full[buf], lead);
          }
        }
        // every product issued above has completed before TMEM is released
        ptx::mma_commit_pair(&S.drain, lead);
        ptx::mbar_drain(&S.drain, 0);
      }
    }
    if constexpr (kMode == kGateBwd) {
      if (warp == 3 && ptx::elect_one()) {
        // ---------------------------------------------------------- carrier
        const int mine = pair < sh.units ? (sh.units - 1 - pair) / n_pairs + 1 : 0;   // tiles of this pair
        auto place = [&](int q, int& col, int& row) {   // of the q-th 64 columns
          const Unit w = unit_of<kNarrow>(p, sh, pair + (q >> 2) * n_pairs, team, teams);
          col = w.n * kTile + (q & 3) * 64;
          row = w.m * kTile + static_cast<int>(rank) * kHalf;
        };
        auto fetch = [&](int q) {
          int col, row;
          place(q, col, row);
          uint64_t* bar = &S.in_full[0][q & 1];
          ptx::mbar_arrive_expect_tx(bar, 2 * kBoxBytes);
          ptx::tma_load_2d(S.out[q & 1][0], &maps.in, bar, col, row);
          ptx::tma_load_2d(S.out[q & 1][1], &maps.in2, bar, col, row);
        };
        const int n = 4 * mine;
        int issued = n < 2 ? n : 2;
        for (int q = 0; q < issued; ++q) fetch(q);
        for (int q = 0; q < n; ++q) {
          if (!ptx::mbar_wait(&S.written[q & 1], (q >> 1) & 1, abort_flag, kWaitLimitNs)) break;
          int col, row;
          place(q, col, row);
          if (col < p.N && row < p.M) {
            ptx::tma_store_2d(&maps.out, S.out[q & 1][0], col, row);
            ptx::tma_store_2d(&maps.out2, S.out[q & 1][1], col, row);
          }
          ptx::bulk_commit();
          if (issued < n) {
            ptx::bulk_wait_read<0>();
            fetch(issued++);
          }
        }
        // after a timeout: no copy is left under way
        for (int q = issued > 2 ? issued - 2 : 0; q < issued; ++q)
          ptx::mbar_drain(&S.in_full[0][q & 1], (q >> 1) & 1);
        ptx::bulk_wait_read<0>();
      }
    }
    if (kNarrow && teams > 1) {
      __syncwarp();
      ptx::cluster_sync();   // the other pairs' sums are there
    }
  } else {
    // ------------------------------------------------------------ epilogue
    if constexpr (!kOne) ptx::regs_inc<kRegsEpi>();
    const int wg = (warp - 4) >> 2;
    const int lane = threadIdx.x & 31;
    const int rc = (warp & 3) * 32 + lane;   // row of this CTA's half tile
    const bool leader = (threadIdx.x & 127) == 0;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t bar_empty[2] = {ptx::cluster_addr(&S.tm_empty[0], lead), ptx::cluster_addr(&S.tm_empty[1], lead)};
    uint8_t* const box[2] = {S.out[wg][0], S.out[wg][Sm::kBoxes - 1]};
    auto meet = [&] { asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory"); };
    bool met = false;     // teams: the barrier behind the other pairs' sums has been passed
    uint32_t taken = 0;   // tiles that took something in; of the last, both boxes' loads may be under way
    uint32_t tile = 0, sent = 0;
    bool ok = true;
    Unit w;
    for (int i = 0; ok && next(i, w); ++i) {
      const int M = kMode == kGrads ? p.sub[w.sub].M : p.M, N = kMode == kGrads ? p.sub[w.sub].N : p.N;
      const CUtensorMap* to = kMode == kGrads ? &maps.grad_out(w.sub) : &maps.out;
      const bool takes =
          (kMode == kDz || kMode == kGateBwd || (kMode == kLin && p.has_in && w.split < 0)) && teams == 1;
      const int row0 = w.m * kTile + static_cast<int>(rank) * kHalf;   // first row of this CTA
      // first column of this warpgroup; kGateBwd: of its 32 in every 64
      const int n0 = w.n * kTileN<kMode, kNarrow> + wg * (kMode == kGateBwd ? 32 : kTileN<kMode, kNarrow> / 2);
      // what the epilogue reads, into the boxes that it will leave from
      auto fetch = [&](int s, int col) {
        ptx::mbar_arrive_expect_tx(&S.in_full[wg][s], kBoxBytes);
        ptx::tma_load_2d(box[s], &maps.in, &S.in_full[wg][s], col, row0);
      };
      auto fetched = [&](int s) {
        return ptx::mbar_wait(&S.in_full[wg][s], (taken - 1) & 1, abort_flag, kWaitLimitNs);
      };
      // kGateBwd: the exponents of this row's groups of the c-th 64 columns, u's above g's
      auto exponents = [&](int c) {
        if (n0 + c * 64 >= p.N || row0 + rc >= p.M) return 0x7f007fu;
        const uint8_t* e = p.exps + (n0 / kGroup + c * 2) * p.exp_rows + row0 + rc;
        return __ldg(e) | static_cast<uint32_t>(__ldg(e + static_cast<int64_t>((p.N + kGroup - 1) / kGroup) * p.exp_rows)) << 16;
      };
      uint32_t exps = 0;
      if constexpr (kMode == kGateBwd) exps = exponents(0);
      if (kMode != kGateBwd && takes) {
        if (leader) {
          ptx::bulk_wait_read<0>();   // the boxes' last results have left
          fetch(0, n0);
          if (!kNarrow) fetch(1, n0 + 64);
        }
        ++taken;
      }
      // the tile's bias, read by all rows from shared memory (a load per 32 columns on
      // its way from DRAM to every thread cost a lone tile 2.5 us)
      if constexpr (kMode == kLin || kMode == kDz) {
        if (p.bias && teams == 1) {
          const int i = threadIdx.x & 127;
          if (!kNarrow || i < 64) S.bias[wg][i] = n0 + i < p.N ? __ldg(p.bias + n0 + i) : 0.f;
        }
      }
      // the accumulator: 128 columns as packed pairs where chunks are added up
      uint64_t z[kOne ? 1 : kHalf / 2];
      if constexpr (!kOne) {
#pragma unroll 1
        for (int k = 0; ok && k < w.nk; k += kChunk) {
          const uint32_t buf = tile & 1;
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(&S.tm_full[buf], (tile / 2) & 1, abort_flag, kWaitLimitNs))) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          ++tile;
          const uint32_t tm = tmem + lane_off + buf * kCols + wg * kHalf;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            ptx::tmem_ld32(tm + c * 32, x);
            ptx::tmem_wait_ld_of(x);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              z[c * 16 + e] = k == 0 ? pair_at(x, e) : ptx::add2(z[c * 16 + e], pair_at(x, e));
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster(bar_empty[buf]);
        }
      } else {
        ok = ptx::mbar_wait(&S.tm_full[tile & 1], (tile / 2) & 1, abort_flag, kWaitLimitNs);
      }
      // a warpgroup has barriers of its own and gives up as a whole; where pairs share a
      // tile the two meet on their way (the cluster's barrier, kDz's sums) and do so together
      ok = kNarrow && teams > 1 ? ptx::all_of<kEpiThreads>(4, ok) : ptx::all_of_128(wg + 1, ok);
      if (!ok) break;
      const uint32_t buf = tile & 1;
      const uint32_t tm =
          tmem + lane_off + buf * kCols + wg * (kMode == kGate || kNarrow ? 64 : kMode == kGateBwd ? 32 : kHalf);
      if constexpr (kOne) {
        ptx::tc_fence_after();
        ++tile;
      }
      auto release = [&] {   // the whole accumulator has been read
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(bar_empty[buf]);
      };

      if constexpr (kNarrow) {
        if (teams > 1) {
          // this row's sums, 16 bytes at a time, to where the stages were
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t y[32];
            ptx::tmem_ld32(tm + c * 32, y);
            ptx::tmem_wait_ld_of(y);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(S.a[0] + team_place(rc, wg * 16 + c * 8 + q)) =
                  make_uint4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
          }
          __syncwarp();
          ptx::cluster_sync();
          met = true;
          // this pair's part of the rows, four at a time per warp, four columns per lane
          const int rows = kHalf / teams, c0 = w.n * kHalf + lane * 4;
          const bool in_n = c0 < p.N;
          uint64_t b0 = 0, b1 = 0;
          if ((kMode == kLin || kMode == kDz) && p.bias && in_n) {
            const ulonglong2 v = __ldg(reinterpret_cast<const ulonglong2*>(p.bias + c0));
            b0 = v.x;
            b1 = v.y;
          }
          float4 sums = make_float4(0.f, 0.f, 0.f, 0.f);   // kDz: of the rows of a group of 32
#pragma unroll 1
          for (int i0 = (warp - 4) * 4; i0 < rows; i0 += 32) {
            uint64_t x[4][2] = {};
#pragma unroll 2
            for (int k = 0; k < teams; ++k) {
              const uint32_t from = ptx::cluster_addr(S.a[0], static_cast<uint32_t>(2 * k) + rank);
              ulonglong2 y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = ptx::lds128u_cluster(from + team_place(team * rows + i0 + j, lane));
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                x[j][0] = ptx::add2(x[j][0], y[j].x);
                x[j][1] = ptx::add2(x[j][1], y[j].y);
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = row0 + team * rows + i0 + j;
              const bool inside = row < p.M && in_n;
              if constexpr (kMode == kLin || kMode == kDz) {
                uint2 q = make_uint2(0, 0);
                if (p.in && inside) q = *reinterpret_cast<const uint2*>(p.in + row * p.ld_in + c0);
                const uint64_t y[2] = {ptx::f2(lo16(q.x), hi16(q.x)), ptx::f2(lo16(q.y), hi16(q.y))};
                x[j][0] = ptx::add2(x[j][0], b0);
                x[j][1] = ptx::add2(x[j][1], b1);
                with_act(p.act, [&](auto t) {
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    if constexpr (kMode == kLin) {
                      x[j][e] = ptx::add2(act_2<decltype(t)::value>(x[j][e]), y[e]);
                    } else {
                      uint64_t slope;
                      act_slope_2<decltype(t)::value>(x[j][e], slope);
                      x[j][e] = ptx::mul2(y[e], slope);
                    }
                  }
                });
              }
              float v[4];
              ptx::unf2(x[j][0], v[0], v[1]);
              ptx::unf2(x[j][1], v[2], v[3]);
              if (inside) {
                *reinterpret_cast<uint2*>(p.out + row * p.ld_out + c0) =
                    make_uint2(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]));
                sums.x += v[0]; sums.y += v[1]; sums.z += v[2]; sums.w += v[3];
              }
            }
            if (kMode == kDz && p.colsum) {   // the eight warps have done 32 rows
              float4* part = reinterpret_cast<float4*>(S.out[0][0]);   // [8][32]
              part[(warp - 4) * 32 + lane] = sums;
              sums = make_float4(0.f, 0.f, 0.f, 0.f);
              asm volatile("bar.sync 4, %0;" ::"n"(kEpiThreads) : "memory");
              const int group = (row0 + team * rows + i0) / 32;
              if (warp == 4 && in_n && group * 32 < p.M) {
                float4 s = part[lane];
#pragma unroll
                for (int k = 1; k < 8; ++k) {
                  const float4 y = part[k * 32 + lane];
                  s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
                }
                *reinterpret_cast<float4*>(p.colsum + static_cast<int64_t>(group) * p.N + c0) = s;
              }
              asm volatile("bar.sync 4, %0;" ::"n"(kEpiThreads) : "memory");
            }
          }
          break;   // the one tile there is
        }
      }
      if constexpr (kPlain || kMode == kDz) {
        // 32 columns at a time, read from TMEM while those before go out.  (One copy of
        // the code: a kernel of one tile per CTA pays for every instruction's way here.)
        uint32_t raw[32];
        if constexpr (kOne) {
          ptx::tmem_ld32(tm, raw);
          ptx::tmem_wait_ld_of(raw);
        }
        constexpr int kUnroll = kOne ? 1 : 4, kLast = kNarrow ? 1 : 3;
#pragma unroll kUnroll
        for (int c = 0; c <= kLast; ++c) {
          uint64_t x[16];
          if constexpr (kOne) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = pair_at(raw, e);
            if (c < kLast) ptx::tmem_ld32(tm + (c + 1) * 32, raw);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = z[c * 16 + e];
          }
          const int c0 = n0 + c * 32, b = c >> 1, half = c & 1;
          if (kPlain && w.split >= 0) {
            const int64_t tile_id = static_cast<int64_t>(w.split) * (sh.mt * sh.nt - p.whole) + w.tile - p.whole;
            float* blk = p.acc + tile_id * (kTile * kTile) + (static_cast<int>(rank) * kHalf + rc) * kTile + wg * kHalf;
            ulonglong2* ap = reinterpret_cast<ulonglong2*>(blk + c * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q) ap[q] = make_ulonglong2(x[2 * q], x[2 * q + 1]);
          } else {
            uint32_t o[16];
            if (half == 0) {
              if (takes) {
                ok = fetched(b);
              } else {
                if (leader) ptx::bulk_wait_read<kNarrow || Sm::kBoxes == 1 ? 0 : 1>();   // this box's last store
                meet();
              }
            }
            if constexpr (kMode == kLin || kMode == kDz) {
              uint32_t in[16];
              if (takes) get64(box[b], rc, half, in);
              if (p.bias) {
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const ulonglong2 bv = ptx::lds128u(&S.bias[wg][c * 32 + 2 * e]);
                  x[e] = ptx::add2(x[e], bv.x);
                  x[e + 1] = ptx::add2(x[e + 1], bv.y);
                }
              }
              if constexpr (kMode == kLin) {
                if (p.act != TPK_ACT_NONE)
                  with_act(p.act, [&](auto t) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = act_2<decltype(t)::value>(x[e]);
                  });
                if (takes)
#pragma unroll
                  for (int e = 0; e < 16; ++e) x[e] = ptx::add2(x[e], ptx::f2(lo16(in[e]), hi16(in[e])));
              } else {
                with_act(p.act, [&](auto t) {
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    uint64_t slope;
                    act_slope_2<decltype(t)::value>(x[e], slope);
                    x[e] = ptx::mul2(ptx::f2(lo16(in[e]), hi16(in[e])), slope);
                  }
                });
              }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float lo, hi;
              ptx::unf2(x[e], lo, hi);
              o[e] = ptx::pack_bf16x2(lo, hi);
            }
            if (kMode == kDz && p.colsum) {
              float v[32];
              const bool inside = row0 + rc < p.M;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                ptx::unf2(x[e], v[2 * e], v[2 * e + 1]);
                if (!inside) v[2 * e] = v[2 * e + 1] = 0.f;
              }
              const float sum = column_sums(v, lane);
              if (row0 + (warp & 3) * 32 < p.M && c0 + lane < p.N)
                p.colsum[static_cast<int64_t>(row0 / 32 + (warp & 3)) * p.N + c0 + lane] = sum;
            }
            put64(box[b], rc, half, o);
            if (half == 1) {
              ptx::fence_async_shared();
              meet();
              if (leader) {
                if (c0 - 32 < N && row0 < M) ptx::tma_store_2d(to, box[b], c0 - 32, row0);
                ptx::bulk_commit();
              }
            }
          }
          if constexpr (kOne) {
            if (c < kLast) ptx::tmem_wait_ld_of(raw);
            if (c == kLast - 1) release();
          }
        }
      } else if constexpr (kMode == kGate) {
        // columns [0, 64) of this warpgroup: g at 0, u at 128 of the accumulator
        uint32_t a[2][16], u16[2][16];
        auto take_box = [&] {   // its last store has left
          if (leader) ptx::bulk_wait_read<0>();
          meet();
        };
        auto send = [&](const CUtensorMap* to) {
          ptx::fence_async_shared();
          meet();
          if (leader) {
            if (n0 < p.N && row0 < p.M) ptx::tma_store_2d(to, box[0], n0, row0);
            ptx::bulk_commit();
          }
        };
        if (p.save) take_box();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t g[32], up[32];
          ptx::tmem_ld32(tm + half * 32, g);
          ptx::tmem_ld32(tm + kHalf + half * 32, up);
          ptx::tmem_wait_ld_of(g);
          ptx::tmem_wait_ld_of(up);
          if (half == 1) release();
          if (p.save) {
            const uint32_t eg = largest_exponent(g), eu = largest_exponent(up);
            if (n0 + half * kGroup < p.N && row0 + rc < p.M) {
              const int64_t groups = (p.N + kGroup - 1) / kGroup;
              uint8_t* e = p.exps + (n0 / kGroup + half) * p.exp_rows + row0 + rc;
              e[0] = static_cast<uint8_t>(eg);
              e[groups * p.exp_rows] = static_cast<uint8_t>(eu);
            }
            const uint64_t sg = both(group_scale(eg)), su = both(group_scale(eu));
            uint32_t o[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float lo, hi;
              ptx::unf2(ptx::mul2(pair_at(g, e), sg), lo, hi);
              o[e] = ptx::pack_f16x2(lo, hi);
              ptx::unf2(ptx::mul2(pair_at(up, e), su), lo, hi);
              u16[half][e] = ptx::pack_f16x2(lo, hi);
            }
            put64(box[0], rc, half, o);
            if (half == 1) send(&maps.out2);
          }
          with_act(p.act, [&](auto t) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float lo, hi;
              ptx::unf2(ptx::mul2(act_2<decltype(t)::value>(pair_at(g, e)), pair_at(up, e)), lo, hi);
              a[half][e] = ptx::pack_bf16x2(lo, hi);
            }
          });
        }
        if (p.save) {
          take_box();
          put64(box[0], rc, 0, u16[0]);
          put64(box[0], rc, 1, u16[1]);
          send(&maps.out3);
        }
        take_box();
        put64(box[0], rc, 0, a[0]);
        put64(box[0], rc, 1, a[1]);
        send(&maps.out);
      } else {
        // kGateBwd: 32 of 64 columns at a time, g and u in the two boxes of a place
        uint32_t raw[32];
        ptx::tmem_ld32(tm, raw);
        ptx::tmem_wait_ld_of(raw);
#pragma unroll 1
        for (int c = 0; c < 4; ++c, ++sent) {
          uint64_t x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = pair_at(raw, e);
          const uint64_t sg = both(group_unscale(exps & 0xff)), su = both(group_unscale(exps >> 16));
          if (c < 3) {
            ptx::tmem_ld32(tm + (c + 1) * 64, raw);
            exps = exponents(c + 1);
          }
          const int s = static_cast<int>(sent & 1);
          ok = ptx::mbar_wait(&S.in_full[0][s], (sent >> 1) & 1, abort_flag, kWaitLimitNs) && ok;
          uint32_t g16[16], u16[16];
          get64(S.out[s][0], rc, wg, g16);
          get64(S.out[s][1], rc, wg, u16);
          with_act(p.act, [&](auto t) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t g = ptx::mul2(ptx::unpack_f16x2(g16[e]), sg);
              const uint64_t u = ptx::mul2(ptx::unpack_f16x2(u16[e]), su);
              const uint64_t da = x[e];
              uint64_t slope;
              const uint64_t v = act_slope_2<decltype(t)::value>(g, slope);
              float lo, hi;
              ptx::unf2(ptx::mul2(ptx::mul2(da, u), slope), lo, hi);
              g16[e] = ptx::pack_bf16x2(lo, hi);
              ptx::unf2(ptx::mul2(da, v), lo, hi);
              u16[e] = ptx::pack_bf16x2(lo, hi);
            }
          });
          put64(S.out[s][0], rc, wg, g16);
          put64(S.out[s][1], rc, wg, u16);
          ptx::fence_async_shared();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&S.written[s]);
          if (c < 3) ptx::tmem_wait_ld_of(raw);
          if (c == 2) release();
        }
      }
      if (takes) ok = ptx::all_of_128(wg + 1, ok);   // a load that gave up
    }
    if (kNarrow && teams > 1 && !met) {   // gave up before
      __syncwarp();
      ptx::cluster_sync();
    }
    if (kMode != kGateBwd && leader) {
      // loads that nobody waited for (after a timeout) have arrived before the CTA leaves
      for (int s = 0; s < (kNarrow ? 1 : 2); ++s)
        if (taken) ptx::mbar_drain(&S.in_full[wg][s], (taken - 1) & 1);
      ptx::bulk_wait_read<0>();   // (what is still on its way out is out when the kernel is done)
    }
  }
  // The cluster's CTAs leave together: nothing signals or reads a CTA that has
  // gone.  After a timeout in any the stages' copies are waited for first.
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0 && S.abort_flag)
    for (uint32_t i = 0; i < size; ++i) ptx::st_cluster(&S.abort_flag, i, 1);
  ptx::cluster_sync();
  if (S.abort_flag) {
    if (threadIdx.x == 0) {
      if (p.err) *p.err = TPK_E_TIMEOUT;
      if (rank == 0)
        for (uint32_t i = S.issued > kStages ? S.issued - kStages : 0; i < S.issued; ++i)
          ptx::mbar_drain(&S.full[i % kStages], (i / kStages) & 1);
    }
    __syncwarp();
    ptx::cluster_sync();
  }
  ptx::tc_fence_after();
  if (warp == 2) ptx::tmem_dealloc_pair(tmem, 2 * kCols);
  if (p.early) ptx::dependency_wait();
}

// ---- host -------------------------------------------------------------------------
// A row-major bf16 matrix whose rows lie ld elements apart.
struct Mat {
  const void* p;
  int64_t rows, cols, ld;
};
inline int map_of(CUtensorMap* m, const Mat& a, int box_rows) { return make_map_2d(m, a.p, a.rows, a.cols, a.ld, box_rows); }

// Row stride of the library's own buffers: rows that start on 128 bytes take the
// TMA one line per box and row, others two.
inline int64_t own_stride(int64_t cols) { return (cols + 63) / 64 * 64; }

inline int64_t tiles_of(int64_t M, int64_t N) { return (M + kTile - 1) / kTile * ((N + kTile - 1) / kTile); }
// Workspace of a product that may be split over K.
inline size_t acc_bytes(const Plan& p) {
  return static_cast<size_t>(p.split.tail) * p.split.splits * kTile * kTile * 4;
}
inline size_t acc_bytes(int64_t M, int64_t N, int64_t K) { return acc_bytes(plan_of(M, N, K)); }
// Rows of the exponents that kGate keeps, and their bytes.
inline int64_t exp_rows(int64_t N) { return (N + 127) / 128 * 128; }
inline size_t exp_bytes(int64_t N, int64_t I) { return static_cast<size_t>((I + kGroup - 1) / kGroup * 2 * exp_rows(N)); }

// Kernel launch in clusters; after: the stream's last kernel is this library's, of
// the same call, and this one may start under its end (it waits for it itself).
template <typename... Args, typename... Given>
int launch_kernel(void (*kern)(Args...), dim3 grid, int threads, size_t smem, int cluster, bool after, cudaStream_t s,
                  Given... given) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (after) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return launched(cudaLaunchKernelEx(&cfg, kern, static_cast<Args>(given)...));
}

// One of a backward's products: out[M, N] = A B over K.
struct Grad {
  Mat a;          // dz: [M, K], or [K, M] for a weight's gradient (amn)
  bool amn;
  Mat b;          // [K, N]
  Mat out;
};
// Plans up to three of them as one launch; false if one after the other is quicker
// (each pays about 4 us for its start and end), or a sum is too long for one piece.
inline bool grads_plan(const Grad* g, int n, Params* p) {
  int64_t units = 0, work = 0, longest = 0, last = 0;
  double apart = 0.0;
  int order[3] = {0, 1, 2};
  auto k_of = [&](int i) { return ((g[i].amn ? g[i].a.rows : g[i].a.cols) + 63) / 64; };
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && k_of(order[j]) > k_of(order[j - 1]); --j) {
      const int x = order[j];
      order[j] = order[j - 1];
      order[j - 1] = x;
    }
  for (int i = 0; i < 3; ++i) p->sub[i] = Sub{0, 0, 1, 0, 0, 0};
  for (int i = 0; i < n; ++i) {
    const Grad& x = g[order[i]];
    const int64_t k = k_of(order[i]), mt = (x.out.rows + kTile - 1) / kTile, nt = (x.out.cols + kHalf - 1) / kHalf;
    if (k > kChunk || mt * nt > 16 * kPairs) return false;
    p->sub[i] = Sub{static_cast<int32_t>(x.out.rows), static_cast<int32_t>(x.out.cols), static_cast<int32_t>(k),
                    x.amn, static_cast<int32_t>(mt), static_cast<int32_t>(nt)};
    units += mt * nt;
    work += mt * nt * k;
    longest = k > longest ? k : longest;
    last = k;
    apart += plan_of(x.out.rows, x.out.cols, k * 64).us + 4.0;
  }
  // the busiest pair: its share and one tile more, or one of the longest sums
  const int64_t share = (work + kPairs - 1) / kPairs + last;
  const int64_t stages = units <= kPairs ? longest : longest + last > share ? longest + last : share;
  return (units <= kPairs / 2 ? 0.14 : 0.2) * static_cast<double>(stages) + 1.1 + 4.0 < apart;
}
// They, as planned (order of p.sub).
int grads_product(const Grad* g, int n, Params& p, bool after, int32_t* err, cudaStream_t s);

template <int kMode, bool kOne, bool kNarrow = false>
int launch(const Maps& maps, const Params& p, bool after, cudaStream_t s) {
  constexpr auto kern = product_kernel<kMode, kOne, kNarrow>;
  static PerContext<int> rec;
  int unused = 0;
  const int st = guarded([&] { return rec.get(&unused, [](int*) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return TPK_E_CUDA;
    // setmaxnreg waits for registers the CTA was not launched with
    if (!kOne && fa.numRegs * kThreads < kRegsNeeded) return TPK_E_UNSUPPORTED;
    return cuda_status(
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes<kMode>)));
  }); });
  if (st != TPK_OK) return st;
  int units = shape_of<kMode, kNarrow>(p).units;
  if (kMode == kGrads) {
    units = 0;
    for (const Sub& x : p.sub) units += x.mt * x.nt;
  }
  int clusters = num_sms() / 2;
  clusters = clusters < 1 ? 1 : clusters;
  clusters = clusters < units || p.teams > 1 ? (p.teams > 1 ? units : clusters) : units;
  const int size = 2 * p.teams;
  return launch_kernel(kern, dim3(static_cast<unsigned>(size * clusters)), kThreads, kSmemBytes<kMode>, size, after, s,
                       maps, p);
}

// Products of linear.cu that the feed-forward block uses too.  acc: acc_bytes;
// after: as in launch_kernel.
// y = act(x w^T + bias) + residual (residual.p may be nullptr)
int linear_product(const Mat& x, const Mat& w, const float* bias, int act, const Mat& residual, const Mat& y,
                   float* acc, bool after, int32_t* err, cudaStream_t s);
// dx = dz w, up to join_left of *left
int input_product(const Mat& dz, const Mat& w, const Mat& dx, float* acc, bool after, int32_t* err, cudaStream_t s,
                  Params* left);
// dw = dz^T x, up to join_left of *left; `before`: the stream's last kernel, a product of which it needs nothing
int weight_product(const Mat& dz, const Mat& x, const Mat& dw, float* acc, const Params& before, int32_t* err,
                   cudaStream_t s, Params* left);
// The sums of a product's split tiles, where it has any.
int join_left(const Params& left, const Mat& out, cudaStream_t s);

}  // namespace product
}  // namespace tpk
