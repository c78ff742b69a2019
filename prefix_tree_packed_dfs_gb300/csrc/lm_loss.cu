// Softmax cross entropy over a large vocabulary, fused with the output
// projection and never keeping the logits, and its gradients.
//
//   z[f, v] = scale * h[f] . w[v],   lse[f] = ln sum_v exp z[f, v]
//   loss[f] = lse[f] - z[f, target[f]]
//   dz[f, v] = dloss[f] * scale * (exp(z[f, v] - lse[f]) - (v == target[f]))
//   dh[f] = sum_v dz[f, v] w[v],     dw[v] = sum_f dz[f, v] h[f]
// A position whose target lies outside [0, V) has no loss: its loss, lse and
// dh are zero and its row of h reaches nothing (not even as 0 * NaN).  The
// positions that have a target are first gathered into consecutive rows, so
// the others cost no products either; forwards too small for that to pay
// (use_direct, use_few) compute them and drop them.
//
// Everything is one matrix product with four epilogues (kFwd, kDz, kDh, kDw):
//   kFwd  h w^T: each row's running (maximum, sum of exponentials) over a run
//         of vocabulary tiles and the target's score; joined by a small kernel
//   kDz   h w^T again for one piece of the vocabulary: dz in bf16
//   kDh   dz w over the piece, accumulated over the pieces in fp32
//   kDw   dz^T h: the piece's rows of dw
// The vocabulary is cut into pieces so that dz of one piece fits the
// workspace (kDzBytes).  dz enters its products as bf16 (as the score
// gradients do in the attention backward): a relative rounding of 2^-8 at
// most, the size of the outputs' own.  At a target of probability near 1 the
// element is the small difference exp(z - lse) - 1, which carries any error of
// z against lse whole; so kDz computes the very scores of kFwd (the same
// chunks of K in the same order), and z - lse is formed before anything is
// rounded: what is left is the rounding of lse itself, |lse| 2^-24.
//
// The product: 256 x 256 tiles on a pair of CTAs (tcgen05 cta_group::2, each
// CTA holds 128 rows of A, 128 rows of B and its 128 rows of the result), 64
// elements of K per stage, stages filled by TMA, two accumulators of 256 TMEM
// columns so that a tile's epilogue runs under the next tile's products.
// One CTA with a 128 x 256 tile would load 96 bytes of operands per cycle and
// SM at full tensor rate; the pair loads 64.
// The tensor core adds to its fp32 accumulator with truncation, a bias towards
// zero that grows with the number of steps of 16 (measured: a score of 6 at
// width 4,096 came out 2.5e-5 low; a gradient summed over 200,000 terms of one
// sign 1.2e-3).  So an accumulation stops after kChunkOf stages and the epilogue
// adds the chunks up in registers with rounding to nearest: 512 elements for
// the scores, 2,048 for dh and dw, whose results are rounded to bf16 (there
// 1e-5 is left; with 512 the products took 1 to 2% longer).
// Warps of a CTA: 0 TMA producer, 1 MMA issuer (of the pair's first CTA), 2
// TMEM owner, 4-11 epilogue (two warpgroups, 128 columns each).  At widths
// below about 1,000 the epilogue is what a tile waits for: its arithmetic is
// on packed fp32 pairs, a chunk of 32 columns is read from TMEM while the one
// before is worked on, and bf16 results (dz, dw) leave through shared memory
// by TMA (stores of 64 bytes per row straight from the registers took 1.5x the
// time: dz of 9,441 rows, width 552, 61,282 ids 855 us against 579).  CTAs are
// persistent and walk the tiles in panels of 8 columns of tiles, so the pairs
// running together share rows of A and of B in L2.
// What bounds it: the tensor pipe, busy 98% of the forward's cycles and 90-94%
// of the others' (8,192 rows, width 2,048, 32,000 ids: forward 516 us, 2,080
// TFLOP/s; dz 564, dh 584, dw 572 us); in long runs the power limit.
#include <type_traits>

#include "pair.cuh"
#include "rowwise.cuh"

namespace tpk {
namespace {

constexpr int kTile = 256;            // rows and columns of a pair's tile
constexpr int kHalf = 128;            // rows of A / of B a CTA holds
constexpr int kBoxBytes = kHalf * 128;// one stage's operand: 128 x 64 bf16
constexpr int kThreads = 384;
constexpr int kEpiThreads = 256;
constexpr int kPanel = 8;
constexpr int kSplitPairs = 76;       // pairs a split over K aims to fill (two SMs each)
constexpr float kLog2e = 1.4426950408889634f;

enum { kFwd = 0, kDz = 1, kDh = 2, kDw = 3 };

// Stages of 64 elements per accumulation.
template <int kMode>
constexpr int kChunkOf = kMode == kFwd || kMode == kDz ? 8 : 32;
// The epilogue holds 128 columns of a row per thread: the other warps give
// registers to its two warpgroups.
constexpr uint32_t kRegsCtl = 56;
constexpr uint32_t kRegsEpi = 216;
constexpr int kRegsNeeded = 128 * kRegsCtl + 256 * kRegsEpi;

struct LmParams {
  const int32_t* count;     // device: gathered rows; nullptr: n_rows
  int32_t n_rows;
  int32_t V, C;
  int64_t np;               // rows of the padded buffers
  const int32_t* rows;      // gathered row -> position; nullptr: the same
  const int32_t* target;
  const float* lse;
  const float* dloss;
  float scale, scale_log2;
  float2* part;             // kFwd: [2 * chunks][np] (maximum score, sum of exponentials), scores unscaled
  float* zt;                // kFwd: [np] the target's score, unscaled
  int32_t run;              // kFwd: vocabulary tiles per unit
  int32_t v0, vcols, ld_dz; // the piece: first id, ids, row stride of dz
  float* acc;               // kDh: fp32 tiles; kDw: fp32 tiles of a split over K
  int32_t split_most;       // kDh
  int32_t first, last;      // kDh: first / last piece
  __nv_bfloat16* dh;
  __nv_bfloat16* dw;        // kDw without any rows (else through the tensor map)
  int32_t* err;
};

// Splits over K where the tiles alone do not fill the GPU: one round of units
// for a few tiles; otherwise, below four rounds, the split into up to 8 that
// makes the rounds shortest, where it saves a tenth or more (111 tiles in two
// rounds of one against three rounds of a half: 559 -> 471 us, the splits' sum
// included, for dh of 9,441 rows, width 552, 61,282 ids).  `most`: splits with 8 or more stages of K each.
constexpr int kSplitRounds = 4, kSplitMost = 8;
__host__ __device__ inline int splits_for(int64_t tiles, int most) {
  if (tiles <= 0 || tiles > kSplitRounds * kSplitPairs || most <= 1) return 1;
  if (tiles * kSplitMost <= kSplitPairs) {
    const int s = kSplitPairs / static_cast<int>(tiles);
    return s < most ? s : most;
  }
  const int t = static_cast<int>(tiles);
  int best = 1, rounds = (t + kSplitPairs - 1) / kSplitPairs;
  for (int s = 2; s <= kSplitMost && s <= most; ++s) {
    const int r = (t * s + kSplitPairs - 1) / kSplitPairs;
    if (r * best * 10 <= rounds * s * 9) {
      best = s;
      rounds = r;
    }
  }
  return best;
}
__host__ __device__ inline int split_limit(int k_iters) { return k_iters / 8; }
// fp32 tiles that a split product of `tiles` tiles, or of any smaller number
// (the rows are counted on the device), writes.
inline int64_t split_tiles(int64_t tiles) {
  static const int64_t widest = [] {
    int64_t w = 0;
    for (int t = 1; t <= kSplitRounds * kSplitPairs; ++t) {
      const int64_t n = static_cast<int64_t>(t) * splits_for(t, kSplitPairs);
      w = n > w ? n : w;
    }
    return w;
  }();
  const int64_t n = tiles * kSplitMost < kSplitPairs ? kSplitPairs : tiles * kSplitMost;
  return n < widest ? n : widest;
}

// kDz and kDw give one stage's room to the tiles on their way out.
template <int kMode>
struct LmSmem {
  static constexpr bool kOut = kMode == kDz || kMode == kDw;
  static constexpr int kStages = kOut ? 5 : 6;
  static constexpr int kOutBoxes = kOut ? 2 : 0;   // per warpgroup
  uint8_t a[kStages][kBoxBytes];
  uint8_t b[kStages][kBoxBytes];
  uint8_t out[kOut ? 2 * kOutBoxes : 1][kOut ? kBoxBytes : 1024];
  uint64_t full[kStages], empty[kStages];
  uint64_t tm_full[2], tm_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  uint32_t issued;   // stages the producer has filled
};
template <int kMode>
constexpr size_t kLmSmemBytes = sizeof(LmSmem<kMode>) + 1024;
static_assert(kLmSmemBytes<kFwd> <= 227 * 1024 && kLmSmemBytes<kDz> <= 227 * 1024, "shared memory");

// The tiles of one launch.  Unit u covers the column tiles [n0, n0 + n_run) of
// row tile m, and the stages [k0, k0 + nk) of K.
struct Shape {
  int mt, nt, units, splits, k_iters, run;
};
struct Unit {
  int m, n0, n_run, k0, nk, split;
};

template <int kMode>
__device__ __forceinline__ Shape shape_of(const LmParams& p, int count) {
  Shape s;
  const int row_tiles = (count + kTile - 1) / kTile;
  s.splits = 1;
  s.run = 1;
  if constexpr (kMode == kFwd || kMode == kDz) {
    s.mt = row_tiles;
    const int vt = kMode == kFwd ? (p.V + kTile - 1) / kTile : (p.vcols + kTile - 1) / kTile;
    s.run = kMode == kFwd ? p.run : 1;
    s.nt = (vt + s.run - 1) / s.run;
    s.k_iters = (p.C + 63) / 64;
  } else if constexpr (kMode == kDh) {
    s.mt = row_tiles;
    s.nt = (p.C + kTile - 1) / kTile;
    s.k_iters = (p.vcols + 63) / 64;
    s.splits = splits_for(static_cast<int64_t>(s.mt) * s.nt, p.split_most);
  } else {
    s.mt = (p.vcols + kTile - 1) / kTile;
    s.nt = (p.C + kTile - 1) / kTile;
    s.k_iters = (count + 63) / 64;
    s.splits = splits_for(static_cast<int64_t>(s.mt) * s.nt, split_limit(s.k_iters));
  }
  s.units = s.mt * s.nt * s.splits;
  return s;
}

template <int kMode>
__device__ __forceinline__ Unit unit_of(const LmParams& p, const Shape& s, int u) {
  Unit w;
  const int tiles = s.mt * s.nt;
  w.split = u / tiles;
  int t = u - w.split * tiles;
  const int panel = t / (kPanel * s.mt);
  t -= panel * kPanel * s.mt;
  const int width = min(kPanel, s.nt - panel * kPanel);
  w.m = t / width;
  const int n = panel * kPanel + t % width;
  w.n0 = n * s.run;
  w.n_run = 1;
  if constexpr (kMode == kFwd) w.n_run = min(s.run, (p.V + kTile - 1) / kTile - w.n0);
  w.k0 = static_cast<int>(static_cast<int64_t>(s.k_iters) * w.split / s.splits);
  w.nk = static_cast<int>(static_cast<int64_t>(s.k_iters) * (w.split + 1) / s.splits) - w.k0;
  return w;
}

// Columns 2 e and 2 e + 1 of 32 read from TMEM.
__device__ __forceinline__ uint64_t pair_at(const uint32_t (&x)[32], int e) {
  return ptx::f2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
}

// kOne: every tile is a single accumulation, which then need not be held whole
// and goes out while it is read from TMEM (5,003 rows, width 64, 32,000 ids: dz
// 89 us against 100; dw of 4 rows, width 4,096, 131,072 ids: 183 against 208).
template <int kMode, bool kOne>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    lm_product_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                      const __grid_constant__ CUtensorMap tm_out, const LmParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = LmSmem<kMode>;
  constexpr int kStages = Smem::kStages;
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr bool kAmn = kMode == kDw;                      // A stored with M contiguous
  constexpr bool kBmn = kMode == kDh || kMode == kDw;      // B stored with N contiguous
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = ptx::cluster_rank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  volatile int* abort_flag = &S.abort_flag;
  const int count = p.count ? __ldg(p.count) : p.n_rows;
  const Shape sh = shape_of<kMode>(p, count);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&S.full[s], 1);
      ptx::mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&S.tm_full[b], 1);
      ptx::mbar_init(&S.tm_empty[b], 2 * kEpiThreads / 32);   // every epilogue warp of the pair
    }
    ptx::mbar_init(&S.drain, 1);
    S.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc_pair(&S.tmem_base, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // the other CTA's barriers exist
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  if (warp < 4) {
  if constexpr (!kOne) ptx::regs_dec<kRegsCtl>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (ptx::elect_one()) {
      ptx::prefetch_tensormap(&tm_a);
      ptx::prefetch_tensormap(&tm_b);
      uint32_t it = 0;
      bool ok = true;
      for (int u = pair; ok && u < sh.units; u += n_pairs) {
        const Unit w = unit_of<kMode>(p, sh, u);
        for (int j = 0; ok && j < w.n_run; ++j) {
          const int m0 = w.m * kTile + static_cast<int>(rank) * kHalf;
          const int n0 = (w.n0 + j) * kTile + static_cast<int>(rank) * kHalf;
          for (int k = 0; k < w.nk; ++k, ++it) {
            const int st = it % kStages;
            if (it >= kStages && !ptx::mbar_wait(&S.empty[st], (it / kStages - 1) & 1, abort_flag, kWaitLimitNs)) {
              ok = false;
              break;
            }
            if (rank == 0) ptx::mbar_arrive_expect_tx(&S.full[st], 4 * kBoxBytes);
            const uint32_t bar = ptx::cluster_addr(&S.full[st], 0);
            const int kk = (w.k0 + k) * 64;
            if constexpr (kAmn) {
              ptx::tma_load_2d_pair(S.a[st], &tm_a, bar, m0, kk);
              ptx::tma_load_2d_pair(S.a[st] + kBoxBytes / 2, &tm_a, bar, m0 + 64, kk);
            } else {
              ptx::tma_load_2d_pair(S.a[st], &tm_a, bar, kk, m0);
            }
            if constexpr (kBmn) {
              const int y = kMode == kDh ? p.v0 + kk : kk;
              ptx::tma_load_2d_pair(S.b[st], &tm_b, bar, n0, y);
              ptx::tma_load_2d_pair(S.b[st] + kBoxBytes / 2, &tm_b, bar, n0 + 64, y);
            } else {
              ptx::tma_load_2d_pair(S.b[st], &tm_b, bar, kk, kMode == kDz ? p.v0 + n0 : n0);
            }
          }
        }
      }
      S.issued = it;
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer
    if (ptx::elect_one()) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(kTile, kTile, kAmn, kBmn);
      // K step of 16 elements: 32 bytes along a K-major row, 16 rows of 128
      // bytes of an MN-major box (its two 64-column boxes half a stage apart)
      constexpr uint32_t kStepA = kAmn ? 2048 : 32, kStepB = kBmn ? 2048 : 32;
      uint32_t it = 0, tile = 0;
      bool ok = true;
      for (int u = pair; ok && u < sh.units; u += n_pairs) {
        const Unit w = unit_of<kMode>(p, sh, u);
        if (w.nk == 0) continue;
        constexpr int per = kChunkOf<kMode>;
        const int chunks = (w.nk + per - 1) / per;
        for (int j = 0; ok && j < w.n_run * chunks; ++j, ++tile) {
          const uint32_t buf = tile & 1;
          if (tile >= 2 && !ptx::mbar_wait(&S.tm_empty[buf], (tile / 2 - 1) & 1, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const int nk = min(per, w.nk - j % chunks * per);
          for (int k = 0; k < nk; ++k, ++it) {
            const int st = it % kStages;
            if (!ptx::mbar_wait(&S.full[st], (it / kStages) & 1, abort_flag, kWaitLimitNs)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint64_t ad = ptx::sw128_desc(ptx::smem_addr(S.a[st]), kAmn ? kBoxBytes / 2 : 16, 1024);
            const uint64_t bd = ptx::sw128_desc(ptx::smem_addr(S.b[st]), kBmn ? kBoxBytes / 2 : 16, 1024);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              ptx::mma_ss_pair(tmem + buf * kTile, ptx::desc_add(ad, q * kStepA), ptx::desc_add(bd, q * kStepB), idesc,
                               (k > 0 || q > 0) ? 1u : 0u);
            ptx::mma_commit_pair(&S.empty[st]);
          }
          if (ok) ptx::mma_commit_pair(&S.tm_full[buf]);
        }
      }
      // every product issued above has completed before TMEM is released
      ptx::mma_commit_pair(&S.drain);
      ptx::mbar_drain(&S.drain, 0);
    }
  }
  } else {
    // ------------------------------------------------------------ epilogue
    if constexpr (!kOne) ptx::regs_inc<kRegsEpi>();
    const int wg = (warp - 4) >> 2;                     // column half
    const int lane = threadIdx.x & 31;
    const int rc = (warp & 3) * 32 + lane;              // row of this CTA's half tile
    const int r = static_cast<int>(rank) * kHalf + rc;  // row of the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t bar_empty[2] = {ptx::cluster_addr(&S.tm_empty[0], 0), ptx::cluster_addr(&S.tm_empty[1], 0)};
    // the exponent of 2 of a score (kFwd), of z - lse (kDz)
    const float to_2 = kMode == kFwd ? p.scale_log2 : kLog2e;
    const uint64_t k2 = ptx::f2(to_2, to_2), kz = ptx::f2(p.scale, p.scale);
    uint32_t tile = 0;
    int box = 0;   // kDz, kDw: the warpgroup's next box in shared memory
    bool ok = true;
    for (int u = pair; ok && u < sh.units; u += n_pairs) {
      const Unit w = unit_of<kMode>(p, sh, u);
      if (w.nk == 0) {
        // no ids left for this split (kDh); no rows at all: dw is zero
        if (kMode == kDw) {
          const int at = w.m * kTile + r, c0 = w.n0 * kTile + wg * kHalf;
          if (at < p.vcols)
            for (int c = c0; c < min(c0 + kHalf, p.C); c += 8)
              *reinterpret_cast<uint4*>(p.dw + static_cast<int64_t>(p.v0 + at) * p.C + c) = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      const int row = w.m * kTile + r;
      const int64_t tile_id = static_cast<int64_t>(w.split) * sh.mt * sh.nt + w.m * sh.nt + w.n0;
      // per-row inputs
      int tgt = -1;
      float m = -INFINITY, s = 0.f, coef = 0.f, lse = 0.f;
      int64_t pos = row;
      if (kMode != kDw && row < count) {
        pos = p.rows ? __ldg(p.rows + row) : row;
        if (kMode == kFwd || kMode == kDz) tgt = __ldg(p.target + pos);
        if (tgt < 0 || tgt >= p.V) tgt = -1;
        if (kMode == kDz) {
          coef = __ldg(p.dloss + pos) * p.scale;
          lse = __ldg(p.lse + pos);
          tgt -= p.v0;
        }
      }
      for (int j = 0; j < w.n_run; ++j) {
        // the row's 128 columns as packed pairs, chunks of K added up
        uint64_t z[kHalf / 2];
        auto chunk = [&](auto first) {
          const uint32_t buf = tile & 1;
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(&S.tm_full[buf], (tile / 2) & 1, abort_flag, kWaitLimitNs)))
            return false;
          ptx::tc_fence_after();
          ++tile;
          const uint32_t tm = tmem + lane_off + buf * kTile + wg * kHalf;
          if constexpr (decltype(first)::value) {   // every read in flight at once
            uint32_t x[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) ptx::tmem_ld32(tm + c * 32, x[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              ptx::tmem_wait_ld_of(x[c]);
#pragma unroll
              for (int e = 0; e < 16; ++e) z[c * 16 + e] = pair_at(x[c], e);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t x[32];
              ptx::tmem_ld32(tm + c * 32, x);
              ptx::tmem_wait_ld_of(x);
#pragma unroll
              for (int e = 0; e < 16; ++e) z[c * 16 + e] = ptx::add2(z[c * 16 + e], pair_at(x, e));
            }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster(bar_empty[buf]);
          return true;
        };
        if constexpr (!kOne) {
          ok = chunk(std::true_type{});
#pragma unroll 1
          for (int k = kChunkOf<kMode>; ok && k < w.nk; k += kChunkOf<kMode>) ok = chunk(std::false_type{});
        } else {
          ok = ptx::mbar_wait(&S.tm_full[tile & 1], (tile / 2) & 1, abort_flag, kWaitLimitNs);
        }
        // a warpgroup with barriers of its own gives up as a whole
        if (Smem::kOut) ok = ptx::all_of_128(wg + 1, ok);
        if (!ok) break;
        if constexpr (kMode == kFwd) {
          // unscaled scores and their maximum: the differences are exact to a
          // rounding, which products with the scale would not leave them
          const int c0 = (w.n0 + j) * kTile + wg * kHalf;
          if (c0 + kHalf > p.V)
#pragma unroll
            for (int e = 0; e < kHalf / 2; ++e) {
              float lo, hi;
              ptx::unf2(z[e], lo, hi);
              z[e] = ptx::f2(c0 + 2 * e < p.V ? lo : -INFINITY, c0 + 2 * e + 1 < p.V ? hi : -INFINITY);
            }
          if (static_cast<uint32_t>(tgt - c0) < static_cast<uint32_t>(kHalf)) {
            // the target's score, halving the columns by the bits of its place
            uint64_t y[kHalf / 4];
            const int at = tgt - c0;
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = at & 64 ? z[32 + e] : z[e];
#pragma unroll
            for (int half = 16; half > 0; half >>= 1)
#pragma unroll
              for (int e = 0; e < half; ++e) y[e] = at & (2 * half) ? y[half + e] : y[e];
            float lo, hi;
            ptx::unf2(y[0], lo, hi);
            p.zt[row] = at & 1 ? hi : lo;
          }
          float top[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kHalf / 2; ++e) {
            float lo, hi;
            ptx::unf2(z[e], lo, hi);
            top[e & 3] = ptx::max3(top[e & 3], lo, hi);
          }
          const float mn = ptx::max3(top[0], top[1], fmaxf(top[2], top[3]));
          const float ms = mn == -INFINITY ? 0.f : mn;
          const uint64_t neg = ptx::f2(-ms, -ms);
          uint64_t q[4] = {};
#pragma unroll
          for (int e = 0; e < kHalf / 2; ++e) {
            float lo, hi;
            ptx::unf2(ptx::mul2(ptx::add2(z[e], neg), k2), lo, hi);
            q[e & 3] = ptx::add2(q[e & 3], ptx::f2(ptx::ex2(lo), ptx::ex2(hi)));
          }
          float lo, hi;
          ptx::unf2(ptx::add2(ptx::add2(q[0], q[1]), ptx::add2(q[2], q[3])), lo, hi);
          // the tile's sum first: many small terms added one by one onto the
          // large term of an earlier tile would round away
          s = fmaf(s, ptx::ex2((m - ms) * p.scale_log2), lo + hi);
          m = mn;
        } else {
          const int n0 = (w.n0 + j) * kTile + wg * kHalf;   // first column of this warpgroup
          // columns 32 c .. 32 c + 31 on their way out
          auto emit = [&](int c, const uint64_t(&x)[16]) {
            const int c0 = n0 + c * 32;
            if constexpr (kMode == kDz || kMode == kDw) {
              uint32_t o[16];
              if constexpr (kMode == kDz) {
                // z - lse, then the exponent of 2: with lse scaled first, the small
                // difference of a p near 1 would carry that rounding too
                const uint64_t minus = ptx::f2(-lse, -lse), c2 = ptx::f2(coef, coef);
                float d[32];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  float lo, hi;
                  ptx::unf2(ptx::mul2(ptx::fma2(x[e / 2], kz, minus), k2), lo, hi);
                  d[e] = ptx::ex2(lo);
                  d[e + 1] = ptx::ex2(hi);
                }
                if (static_cast<uint32_t>(tgt - c0) < 32u) {
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (tgt - c0 == e) d[e] -= 1.f;
                }
                if (c0 + 32 > p.vcols)
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (c0 + e >= p.vcols) d[e] = 0.f;
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  float lo, hi;
                  ptx::unf2(ptx::mul2(ptx::f2(d[e], d[e + 1]), c2), lo, hi);
                  o[e / 2] = ptx::pack_bf16x2(lo, hi);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  float lo, hi;
                  ptx::unf2(x[e], lo, hi);
                  o[e] = ptx::pack_bf16x2(lo, hi);
                }
              }
              if (kMode == kDz || sh.splits == 1) {
                // out through shared memory: 64 columns per box, in the TMA's
                // swizzle (16-byte piece i of row r at piece i ^ (r % 8))
                uint8_t* stage = S.out[wg * Smem::kOutBoxes + box];
                const bool leader = (threadIdx.x & 127) == 0;
                if ((c & 1) == 0) {
                  if (leader) ptx::bulk_wait_read<Smem::kOutBoxes - 1>();   // this box's last store
                  asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory");
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  *reinterpret_cast<uint4*>(stage + rc * 128 + ((((c & 1) * 4 + q) ^ (rc & 7)) * 16)) =
                      make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                if ((c & 1) == 1) {
                  ptx::fence_async_shared();
                  asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory");
                  const int col = c0 - 32;
                  const int first_row = w.m * kTile + static_cast<int>(rank) * kHalf;
                  const bool inside = kMode == kDz ? col < p.ld_dz : col < p.C && first_row < p.vcols;
                  if (leader) {
                    if (inside) ptx::tma_store_2d(&tm_out, stage, col, kMode == kDw ? p.v0 + first_row : first_row);
                    ptx::bulk_commit();
                  }
                  box = (box + 1) % Smem::kOutBoxes;
                }
              } else {
                float* blk = p.acc + tile_id * (kTile * kTile) + r * kTile + wg * kHalf + c * 32;
                ulonglong2* ap = reinterpret_cast<ulonglong2*>(blk);
#pragma unroll
                for (int q = 0; q < 8; ++q) ap[q] = make_ulonglong2(x[2 * q], x[2 * q + 1]);
              }
            } else {
              float* blk = p.acc + tile_id * (kTile * kTile) + r * kTile + wg * kHalf + c * 32;
              const bool out = p.last && sh.splits == 1;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint64_t v[4] = {x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
                ulonglong2* ap = reinterpret_cast<ulonglong2*>(blk + 8 * q);
                if (!p.first) {
                  const ulonglong2 y0 = ap[0], y1 = ap[1];
                  v[0] = ptx::add2(v[0], y0.x);
                  v[1] = ptx::add2(v[1], y0.y);
                  v[2] = ptx::add2(v[2], y1.x);
                  v[3] = ptx::add2(v[3], y1.y);
                }
                if (!out) {
                  ap[0] = make_ulonglong2(v[0], v[1]);
                  ap[1] = make_ulonglong2(v[2], v[3]);
                } else if (row < count && c0 + 8 * q < p.C) {
                  uint32_t o[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    float lo, hi;
                    ptx::unf2(v[e], lo, hi);
                    o[e] = ptx::pack_bf16x2(lo, hi);
                  }
                  *reinterpret_cast<uint4*>(p.dh + pos * p.C + c0 + 8 * q) = make_uint4(o[0], o[1], o[2], o[3]);
                }
              }
            }
          };
          uint64_t x[16];
          if constexpr (kOne) {
            // 32 columns are read from TMEM while those before go out
            const uint32_t buf = tile & 1;
            const uint32_t tm = tmem + lane_off + buf * kTile + wg * kHalf;
            ptx::tc_fence_after();
            ++tile;
            uint32_t raw[2][32];
            ptx::tmem_ld32(tm, raw[0]);
            ptx::tmem_wait_ld_of(raw[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c < 3) ptx::tmem_ld32(tm + (c + 1) * 32, raw[(c + 1) & 1]);
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = pair_at(raw[c & 1], e);
              emit(c, x);
              if (c < 3) ptx::tmem_wait_ld_of(raw[(c + 1) & 1]);
              if (c == 2) {   // the whole tile has been read
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(bar_empty[buf]);
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = z[c * 16 + e];
              emit(c, x);
            }
          }
        }
      }
      if (kMode == kFwd && ok && row < count)
        p.part[(static_cast<int64_t>(w.n0 / sh.run) * 2 + wg) * p.np + row] = make_float2(m, s);
    }
    if (Smem::kOut) ptx::bulk_wait_all();   // (of the threads that stored)
  }
  // Both CTAs leave together: nothing of the pair signals or reads a CTA that
  // has gone.  After a timeout the stages' copies are waited for first.
  __syncwarp();
  __syncthreads();
  ptx::cluster_sync();
  if (S.abort_flag) {
    if (threadIdx.x == 0) {
      if (p.err) *p.err = TPK_E_TIMEOUT;
      if (rank == 0)
        for (uint32_t i = S.issued > kStages ? S.issued - kStages : 0; i < S.issued; ++i)
          ptx::mbar_drain(&S.full[i % kStages], (i / kStages) & 1);
    }
  }
  __syncwarp();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp == 2) ptx::tmem_dealloc_pair(tmem, 512);
}

// ---- gathering the positions that have a target ------------------------------
// rows[0..count) = those positions, ascending; pos[f] = its row or -1; hc[r] =
// h[rows[r]], rows up to the next multiple of 256 zero.  One launch: a CTA
// takes a run of positions and counts the targets before it itself (every CTA
// reads all of target, a few bytes per position against a row's thousands).
constexpr int kRowsThreads = 512;
constexpr int kRowsBlocks = 304;
constexpr int kRowsLeast = 16;   // positions per CTA

__global__ void __launch_bounds__(kRowsThreads) lm_rows_kernel(const int32_t* __restrict__ target, int N, int V,
                                                               const uint4* __restrict__ h, int vecs, int ld,
                                                               int per, int32_t* __restrict__ rows,
                                                               int32_t* __restrict__ pos, int32_t* __restrict__ count,
                                                               uint4* __restrict__ hc) {
  constexpr int kWarps = kRowsThreads / 32;
  __shared__ int sums[2][kWarps];
  __shared__ int list[kRowsThreads];   // positions with a target of the 512 at hand
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * per;
  const int64_t hi = lo + per < N ? lo + per : N;
  int before = 0, all = 0;
  auto add = [&](int64_t i, int t) {
    const int on = t >= 0 && t < V;
    all += on;
    before += i < lo ? on : 0;
  };
  int64_t i0 = 0;
  if (reinterpret_cast<uintptr_t>(target) % 16 == 0) {
    const int64_t quads = N / 4;
#pragma unroll 4
    for (int64_t q = threadIdx.x; q < quads; q += kRowsThreads) {
      const int4 t = __ldg(reinterpret_cast<const int4*>(target) + q);
      add(4 * q, t.x);
      add(4 * q + 1, t.y);
      add(4 * q + 2, t.z);
      add(4 * q + 3, t.w);
    }
    i0 = 4 * quads;
  }
#pragma unroll 8
  for (int64_t i = i0 + threadIdx.x; i < N; i += kRowsThreads) add(i, __ldg(target + i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 0) {
    sums[0][warp] = before;
    sums[1][warp] = all;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += sums[0][w];
    all += sums[1][w];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *count = all;
  for (int64_t at = lo; at < hi; at += kRowsThreads) {
    __syncthreads();   // sums and list of the step before have been read
    const int64_t i = at + threadIdx.x;
    const int t = i < hi ? __ldg(target + i) : -1;
    const bool on = t >= 0 && t < V;
    const unsigned mask = __ballot_sync(0xffffffffu, on);
    if (lane == 0) sums[0][warp] = __popc(mask);
    __syncthreads();
    int mine = __popc(mask & ((1u << lane) - 1)), n = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      mine += w < warp ? sums[0][w] : 0;
      n += sums[0][w];
    }
    if (i < hi) pos[i] = on ? before + mine : -1;
    if (on) {
      rows[before + mine] = static_cast<int>(i);
      list[mine] = static_cast<int>(i);
    }
    __syncthreads();
    for (int k = warp; k < n; k += kWarps) {
      const uint4* src = h + static_cast<int64_t>(list[k]) * vecs;
      uint4* dst = hc + static_cast<int64_t>(before + k) * ld;
#pragma unroll 4
      for (int c = lane; c < vecs; c += 32) dst[c] = __ldg(src + c);
    }
    before += n;
  }
  const int padded = (all + kTile - 1) / kTile * kTile;
  const int step = static_cast<int>(gridDim.x) * kWarps;
  for (int r = all + static_cast<int>(blockIdx.x) * kWarps + warp; r < padded; r += step)
    for (int c = lane; c < vecs; c += 32) hc[static_cast<int64_t>(r) * ld + c] = make_uint4(0, 0, 0, 0);
}

// w with rows 128 bytes aligned.
__global__ void __launch_bounds__(256) lm_align_kernel(const uint4* __restrict__ w, int V, int vecs, int ld,
                                                       uint4* __restrict__ wc) {
  const int lane = threadIdx.x & 31;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < V;
       r += static_cast<int64_t>(gridDim.x) * 8)
#pragma unroll 4
    for (int c = lane; c < vecs; c += 32) wc[r * ld + c] = __ldg(w + r * vecs + c);
}

// (maximum, sum of exponentials of scale * (score - maximum)) of two sets of scores.
__device__ __forceinline__ float2 merge(float2 a, float2 b, float scale_log2) {
  const float m = fmaxf(a.x, b.x);
  const float ms = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * exp2f((a.x - ms) * scale_log2) + b.y * exp2f((b.x - ms) * scale_log2));
}

// loss and lse of every position: the slots' pairs merged, kRows rows per CTA
// and 256 / kRows threads over the slots of each.  Few rows have many slots
// and few CTAs: 4 rows per CTA there, 32 (coalesced) otherwise.
template <int kRows>
__global__ void __launch_bounds__(256) lm_join_kernel(const float2* __restrict__ part, const float* __restrict__ zt,
                                                      const int32_t* __restrict__ pos,
                                                      const int32_t* __restrict__ target, int N, int V, int slots,
                                                      int64_t np, float scale, float scale_log2,
                                                      float* __restrict__ loss, float* __restrict__ lse) {
  constexpr int kWays = 256 / kRows;
  __shared__ float2 sm[kWays][kRows];
  const int row = threadIdx.x % kRows, w = threadIdx.x / kRows;
  const int i = blockIdx.x * kRows + row;
  int r = -1;
  if (i < N) {
    const int t = __ldg(target + i);
    if (t >= 0 && t < V) r = pos ? __ldg(pos + i) : i;
  }
  float2 x = make_float2(-INFINITY, 0.f);
  if (r >= 0) {
#pragma unroll 4
    for (int k = w; k < slots; k += kWays) x = merge(x, __ldg(part + static_cast<int64_t>(k) * np + r), scale_log2);
  }
  sm[w][row] = x;
  __syncthreads();
#pragma unroll
  for (int o = kWays / 2; o > 0; o >>= 1) {
    if (w < o) sm[w][row] = merge(sm[w][row], sm[w + o][row], scale_log2);
    __syncthreads();
  }
  if (w != 0 || i >= N) return;
  x = sm[0][row];
  const float ln_s = logf(x.y);
  lse[i] = r < 0 ? 0.f : fmaf(x.x, scale, ln_s);
  loss[i] = r < 0 ? 0.f : fmaf(x.x - zt[r], scale, ln_s);
}

// ---- a few positions -----------------------------------------------------------
// Up to kFewRows positions (the log-probability of sampled tokens): one read
// of w, which is all the time there is; a tile of 256 rows of the tensor path
// would be almost empty and its 256-column tiles too few to share out evenly.
// A warp takes a few rows of w at a time and keeps the running (maximum, sum)
// of its rows' scores; the CTA's eight warps merge theirs into one slot.
constexpr int kFewRows = 4;
constexpr int kFewMost = 16384;      // fp32 values of h in shared memory
constexpr int kFewBlocks = 608;      // slots
// Rows of w per warp and step, steps of 256 channels loaded together, CTAs per
// SM.  One position: 27.8 us at 32,000 ids of width 2,048 against 30.9 with
// four rows and four steps; with more positions the sums take the registers.
template <int kN>
struct Few {
  static constexpr int kV = kN == 1 ? 2 : 4;
  static constexpr int kUnroll = kN == 1 ? 8 : 2;
  static constexpr int kPerSm = kN == 1 ? 4 : kN == 2 ? 3 : 2;
};

// A score, 8 channels at a time per lane, then the warp's sum: one order for
// the forward's scores and the backward's targets.
__device__ __forceinline__ uint64_t dot8(uint4 w, ulonglong2 a, ulonglong2 b, uint64_t acc) {
  auto pair = [](uint32_t u) { return ptx::f2(lo16(u), hi16(u)); };
  acc = ptx::fma2(pair(w.x), a.x, acc);
  acc = ptx::fma2(pair(w.y), a.y, acc);
  acc = ptx::fma2(pair(w.z), b.x, acc);
  return ptx::fma2(pair(w.w), b.y, acc);
}
__device__ __forceinline__ uint64_t dot8(uint4 w, uint4 h, uint64_t acc) {
  auto pair = [](uint32_t u) { return ptx::f2(lo16(u), hi16(u)); };
  return dot8(w, make_ulonglong2(pair(h.x), pair(h.y)), make_ulonglong2(pair(h.z), pair(h.w)), acc);
}
__device__ __forceinline__ float dot_sum(uint64_t acc) {
  float lo, hi;
  ptx::unf2(acc, lo, hi);
  float z = lo + hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}

template <int kN>
__global__ void __launch_bounds__(256, Few<kN>::kPerSm)
    lm_few_kernel(const uint4* __restrict__ h, const uint4* __restrict__ w, const int32_t* __restrict__ target, int N,
                  int V, int C, int64_t np, float scale_log2, float2* __restrict__ part, float* __restrict__ zt) {
  constexpr int kFewV = Few<kN>::kV;
  extern __shared__ float4 hs[];     // [kN][C / 8] pairs of float4
  __shared__ float2 sm[8][kN];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vecs = C / 8;
  for (int i = threadIdx.x; i < kN * vecs; i += 256) {
    const uint4 x = i / vecs < N ? __ldg(h + i) : make_uint4(0, 0, 0, 0);
    hs[2 * i] = make_float4(lo16(x.x), hi16(x.x), lo16(x.y), hi16(x.y));
    hs[2 * i + 1] = make_float4(lo16(x.z), hi16(x.z), lo16(x.w), hi16(x.w));
  }
  int tgt[kN];
  float2 st[kN];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    tgt[n] = n < N ? __ldg(target + n) : -1;
    st[n] = make_float2(-INFINITY, 0.f);
  }
  __syncthreads();
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8 * kFewV;
  for (int64_t v0 = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * kFewV; v0 < V; v0 += step) {
    uint64_t acc[kFewV][kN] = {};
#pragma unroll Few<kN>::kUnroll
    for (int c = lane; c < vecs; c += 32) {
      uint4 x[kFewV];
#pragma unroll
      for (int i = 0; i < kFewV; ++i)
        x[i] = v0 + i < V ? __ldg(w + (v0 + i) * vecs + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const ulonglong2 a = ptx::lds128u(hs + 2 * (n * vecs + c)), b = ptx::lds128u(hs + 2 * (n * vecs + c) + 1);
#pragma unroll
        for (int i = 0; i < kFewV; ++i) acc[i][n] = dot8(x[i], a, b, acc[i][n]);
      }
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float z[kFewV], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kFewV; ++i) {
        z[i] = dot_sum(acc[i][n]);
        if (v0 + i >= V) z[i] = -INFINITY;
        if (lane == 0 && n < N && v0 + i < V && v0 + i == tgt[n]) zt[n] = z[i];
        top = fmaxf(top, z[i]);
      }
      const float mn = fmaxf(st[n].x, top);
      const float ms = mn == -INFINITY ? 0.f : mn;
      float s = st[n].y * ptx::ex2((st[n].x - ms) * scale_log2);
#pragma unroll
      for (int i = 0; i < kFewV; ++i) s += ptx::ex2((z[i] - ms) * scale_log2);
      st[n] = make_float2(mn, s);
    }
  }
  if (lane == 0)
#pragma unroll
    for (int n = 0; n < kN; ++n) sm[warp][n] = st[n];
  __syncthreads();
  if (threadIdx.x < N) {
    float2 x = sm[0][threadIdx.x];
    for (int k = 1; k < 8; ++k) x = merge(x, sm[k][threadIdx.x], scale_log2);
    part[static_cast<int64_t>(blockIdx.x) * np + threadIdx.x] = x;
  }
}

// dz of a few positions at their targets, for the scores that lm_few_kernel
// computes: those of the tensor core are truncated, by more than exp(z - lse) - 1
// may be off where the target's probability is near 1.  A warp per position.
__global__ void lm_few_target_kernel(const uint4* __restrict__ h, const uint4* __restrict__ w,
                                     const int32_t* __restrict__ target, const int32_t* __restrict__ pos,
                                     const float* __restrict__ lse, const float* __restrict__ dloss, int v0, int vcols,
                                     int vecs, float scale, int ld_dz, __nv_bfloat16* __restrict__ dz) {
  const int lane = threadIdx.x & 31, f = threadIdx.x >> 5;
  const int r = __ldg(pos + f);
  const int64_t t = __ldg(target + f);
  if (r < 0 || t < v0 || t >= int64_t{v0} + vcols) return;
  uint64_t acc = 0;
#pragma unroll 8
  for (int c = lane; c < vecs; c += 32) acc = dot8(__ldg(w + t * vecs + c), __ldg(h + f * vecs + c), acc);
  const float z = dot_sum(acc);
  if (lane == 0)
    dz[static_cast<int64_t>(r) * ld_dz + (t - v0)] =
        __float2bfloat16_rn(__ldg(dloss + f) * scale * expm1f(fmaf(z, scale, -__ldg(lse + f))));
}

// 8 columns of row r of a product that was split over K: its splits' sums.
__device__ __forceinline__ uint4 sum_splits(const float* __restrict__ acc, int64_t r, int col, int mt, int nt,
                                            int splits) {
  const float* from = acc + ((r / kTile) * nt + col / kTile) * (kTile * kTile) + (r % kTile) * kTile + col % kTile;
  const int64_t step = static_cast<int64_t>(mt) * nt * (kTile * kTile);
  float v[8] = {};
  int s = 0;
  for (; s + 4 <= splits; s += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __ldcg(reinterpret_cast<const float4*>(from + (s + i) * step));
      y[i] = __ldcg(reinterpret_cast<const float4*>(from + (s + i) * step) + 1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[0] += x[i].x; v[1] += x[i].y; v[2] += x[i].z; v[3] += x[i].w;
      v[4] += y[i].x; v[5] += y[i].y; v[6] += y[i].z; v[7] += y[i].w;
    }
  }
  for (; s < splits; ++s) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(from + s * step));
    const float4 y = __ldcg(reinterpret_cast<const float4*>(from + s * step) + 1);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
  return make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]), ptx::pack_bf16x2(v[4], v[5]),
                    ptx::pack_bf16x2(v[6], v[7]));
}

// A warp's share of a row: one 16-byte piece per lane; item = (row, 32 pieces).
// dh of every position that the product's last epilogue has not written:
// zero without a target, the sum of the splits over K where there are any.
__global__ void __launch_bounds__(256) lm_dh_kernel(const float* __restrict__ acc, const int32_t* __restrict__ pos,
                                                    const int32_t* __restrict__ count, int N, int C, int split_most,
                                                    uint4* __restrict__ dh) {
  const int lane = threadIdx.x & 31;
  const int mt = (__ldg(count) + kTile - 1) / kTile, nt = (C + kTile - 1) / kTile;
  const int splits = splits_for(static_cast<int64_t>(mt) * nt, split_most);
  const int vecs = C / 8, parts = (vecs + 31) / 32;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  if (splits == 1) {   // rows without a target alone
    for (int64_t i = first; i < N; i += step)
      if (__ldg(pos + i) < 0)
        for (int c = lane; c < vecs; c += 32) dh[i * vecs + c] = make_uint4(0, 0, 0, 0);
    return;
  }
  for (int64_t it = first; it < static_cast<int64_t>(N) * parts; it += step) {
    const int64_t i = it / parts;
    const int c = static_cast<int>(it % parts) * 32 + lane;
    const int r = __ldg(pos + i);
    if (c < vecs) dh[i * vecs + c] = r < 0 ? make_uint4(0, 0, 0, 0) : sum_splits(acc, r, c * 8, mt, nt, splits);
  }
}

// The piece's rows of dw where its product was split over K.
__global__ void __launch_bounds__(256) lm_dw_kernel(const float* __restrict__ acc, const int32_t* __restrict__ count,
                                                    int v0, int vcols, int C, uint4* __restrict__ dw) {
  const int mt = (vcols + kTile - 1) / kTile, nt = (C + kTile - 1) / kTile;
  const int splits = splits_for(static_cast<int64_t>(mt) * nt, split_limit((__ldg(count) + 63) / 64));
  if (splits == 1) return;
  const int lane = threadIdx.x & 31;
  const int vecs = C / 8, parts = (vecs + 31) / 32;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < static_cast<int64_t>(vcols) * parts;
       it += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t r = it / parts;
    const int c = static_cast<int>(it % parts) * 32 + lane;
    if (c < vecs) dw[(v0 + r) * vecs + c] = sum_splits(acc, r, c * 8, mt, nt, splits);
  }
}

// ---- host ------------------------------------------------------------------------
constexpr int64_t kDzBytes = int64_t{4} << 30;   // dz of one piece

int64_t up(int64_t n, int64_t k) { return (n + k - 1) / k * k; }

// The forward takes h as it is, rows without a target included, where
// gathering costs more than it can save: one tile of rows, or a product of
// about 15 us (the gather takes 8).  The backward always gathers: rows
// without a target must not reach dw.
bool use_direct(int64_t N, int64_t V, int32_t C) {
  return N <= kTile || static_cast<double>(N) * static_cast<double>(V) * C <= 1.2e10;
}

// Rows of h and w that do not start on 64 bytes cost the TMA loads a second
// line each: 1.2 to 1.35x the product's time at widths of 552 and 1,000.
// Gathered rows are laid out aligned; w is copied so where there are enough
// rows to pay for reading and writing it once.
int32_t row_stride(int32_t C) { return C % 32 ? (C + 63) / 64 * 64 : C; }
bool align_w(int64_t N, int32_t C, bool backward) { return C % 32 && N >= (backward ? 2048 : 4096); }

struct LmShape {
  int64_t np;        // N rounded up to whole tiles
  int vt;            // vocabulary tiles
  int run, chunks;   // forward: vocabulary tiles per unit, units per row tile
  int64_t piece;     // backward: ids per piece (a multiple of 256)
  int pieces;
};
LmShape lm_shape(int64_t N, int64_t V) {
  LmShape s;
  s.np = up(N, kTile);
  s.vt = static_cast<int>((V + kTile - 1) / kTile);
  // a unit of several vocabulary tiles keeps its rows' statistics in
  // registers: of the lengths that give every pair 16 units or more, the one
  // whose last round of units is fullest (one tile per unit if none does)
  const int64_t mt = s.np / kTile;
  s.run = 1;
  int64_t best = 0;
  for (int run = 1; run <= 16; ++run) {
    const int64_t units = mt * ((s.vt + run - 1) / run);
    if (run > 1 && units < 16 * kSplitPairs) break;
    const int64_t rounds = (units + kSplitPairs - 1) / kSplitPairs * run;   // tiles the busiest pair does
    if (run == 1 || rounds * 64 <= best * 65) {   // longer runs at up to 1.5%
      best = run == 1 || rounds < best ? rounds : best;
      s.run = run;
    }
  }
  s.chunks = (s.vt + s.run - 1) / s.run;
  int64_t most = kDzBytes / (s.np * 2) / kTile * kTile;
  if (most < 4096) most = 4096;
  s.pieces = static_cast<int>((V + most - 1) / most);
  s.piece = up((V + s.pieces - 1) / s.pieces, kTile);
  s.pieces = static_cast<int>((V + s.piece - 1) / s.piece);
  return s;
}

int few_rows(int64_t N) { return N == 3 ? 4 : static_cast<int>(N); }   // the kernel's kN
bool use_few(int64_t N, int32_t C) { return N <= kFewRows && int64_t{few_rows(N)} * C <= kFewMost; }

struct Carve {
  uint8_t* base;
  size_t at = 0;
  template <typename T>
  T* take(int64_t n) {
    T* p = reinterpret_cast<T*>(base + at);
    at += static_cast<size_t>(up(n * static_cast<int64_t>(sizeof(T)), 1024));
    return p;
  }
};

struct LmWork {
  int32_t *rows, *pos, *count;
  __nv_bfloat16* hc;    // gathered rows of h, row_stride apart; nullptr: none
  __nv_bfloat16* wc;    // aligned copy of w; nullptr: none
  float2* part;
  float* zt;
  __nv_bfloat16* dz;
  float* acc_h;
  float* acc_w;
};
size_t carve(uint8_t* base, int64_t N, int64_t V, int32_t C, bool backward, LmWork* w) {
  const LmShape s = lm_shape(N, V);
  Carve c{base};
  LmWork o{};
  if (backward || !use_direct(N, V, C)) {
    o.rows = c.take<int32_t>(s.np);
    o.pos = c.take<int32_t>(s.np);
    o.count = c.take<int32_t>(1);
    o.hc = c.take<__nv_bfloat16>(s.np * row_stride(C));
    if (align_w(N, C, backward)) o.wc = c.take<__nv_bfloat16>(V * row_stride(C));
  }
  if (!backward) {
    int64_t slots = 2 * static_cast<int64_t>(s.chunks);
    if (use_few(N, C) && slots < kFewBlocks) slots = kFewBlocks;
    o.part = c.take<float2>(slots * s.np);
    o.zt = c.take<float>(s.np);
  } else {
    o.dz = c.take<__nv_bfloat16>(s.np * s.piece);
    const int64_t nt = (C + kTile - 1) / kTile;
    const int64_t th = s.np / kTile * nt, sh = split_tiles(th);
    o.acc_h = c.take<float>((s.pieces > 1 && th > sh ? th : sh) * kTile * kTile);   // one piece: splits alone
    // dw: the tiles of a full piece and of the last one are known here
    const int most = split_limit(static_cast<int>(s.np / 64));
    const int64_t full = s.piece / kTile * nt, rest = ((V - (s.pieces - 1) * s.piece) + kTile - 1) / kTile * nt;
    const int64_t sf = splits_for(full, most), sr = splits_for(rest, most);
    const int64_t tw = (sf > 1 ? full * sf : 0) > (sr > 1 ? rest * sr : 0) ? full * sf : (sr > 1 ? rest * sr : 0);
    if (tw) o.acc_w = c.take<float>(tw * kTile * kTile);
  }
  if (w) *w = o;
  return c.at;
}

// (the row counters of the kernels' last strides stay below 2^31)
bool sizes_ok(int64_t N, int64_t V, int32_t C) {
  return N >= 0 && N < (int64_t{1} << 31) - 8192 && V >= 1 && V < (int64_t{1} << 31) - 4096 && C >= 8 && C % 8 == 0 &&
         C <= (1 << 20);
}

template <int kMode, bool kOne = false>
int launch_product(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& out, const LmParams& p,
                   int64_t most_units, cudaStream_t s) {
  constexpr auto kern = lm_product_kernel<kMode, kOne>;
  static PerContext<int> rec;
  int unused = 0;
  const int st = guarded([&] { return rec.get(&unused, [](int*) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return TPK_E_CUDA;
    // setmaxnreg waits for registers the CTA was not launched with
    if (!kOne && fa.numRegs * kThreads < kRegsNeeded) return TPK_E_UNSUPPORTED;
    return cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(kLmSmemBytes<kMode>)));
  }); });
  if (st != TPK_OK) return st;
  int64_t pairs = num_sms() / 2;
  if (pairs < 1) pairs = 1;
  if (pairs > most_units) pairs = most_units;
  kern<<<static_cast<unsigned>(2 * pairs), kThreads, kLmSmemBytes<kMode>, s>>>(a, b, out, p);
  return cuda_status(cudaGetLastError());
}

template <int kN>
int launch_few(const void* h, const void* w, const int32_t* target, int64_t N, int64_t V, int32_t C, int64_t np,
               float scale_log2, int* slots, const LmWork& k, cudaStream_t s) {
  static PerContext<int> rec;
  const int st = guarded([&] { return set_smem_once(rec, lm_few_kernel<kN>, sizeof(float) * kFewMost); });
  if (st != TPK_OK) return st;
  const int64_t want = (V + 8 * Few<kN>::kV - 1) / (8 * Few<kN>::kV);
  int64_t blocks = int64_t{num_sms()} * Few<kN>::kPerSm;
  blocks = blocks > kFewBlocks ? kFewBlocks : blocks;
  blocks = want < blocks ? want : blocks;
  *slots = static_cast<int>(blocks);
  lm_few_kernel<kN><<<static_cast<unsigned>(blocks), 256, static_cast<size_t>(kN) * C * 4, s>>>(
      static_cast<const uint4*>(h), static_cast<const uint4*>(w), target, static_cast<int>(N), static_cast<int>(V), C,
      np, scale_log2, k.part, k.zt);
  return cuda_status(cudaGetLastError());
}

int64_t grid_for(int64_t warps) {
  const int64_t blocks = (warps + 7) / 8, most = int64_t{num_sms()} * 16;
  return blocks < most ? blocks : most;
}

// rows, pos, count and hc of the positions with a target, and w's aligned copy
int gather_rows(const void* h, const void* wt, const int32_t* target, int64_t N, int64_t V, int32_t C, const LmWork& w,
                cudaStream_t s) {
  int64_t per = (N + kRowsBlocks - 1) / kRowsBlocks;
  per = per < kRowsLeast ? kRowsLeast : per;
  const int ld = row_stride(C) / 8;
  lm_rows_kernel<<<static_cast<unsigned>((N + per - 1) / per), kRowsThreads, 0, s>>>(
      target, static_cast<int>(N), static_cast<int>(V), static_cast<const uint4*>(h), C / 8, ld, static_cast<int>(per),
      w.rows, w.pos, w.count, reinterpret_cast<uint4*>(w.hc));
  const int st = cuda_status(cudaGetLastError());
  if (st != TPK_OK || !w.wc) return st;
  lm_align_kernel<<<static_cast<unsigned>(grid_for(V)), 256, 0, s>>>(static_cast<const uint4*>(wt), static_cast<int>(V),
                                                                     C / 8, ld, reinterpret_cast<uint4*>(w.wc));
  return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace tpk

extern "C" size_t tpk_lm_loss_workspace_bytes(int64_t N, int64_t V, int32_t C, int32_t backward) {
  using namespace tpk;
  if (!sizes_ok(N, V, C) || N == 0) return 0;
  return carve(nullptr, N, V, C, backward != 0, nullptr);
}

extern "C" int tpk_lm_loss(const void* h, const void* w, const int32_t* target, float* loss, float* lse, int64_t N,
                           int64_t V, int32_t C, float scale, void* workspace, size_t ws_bytes, int32_t* dev_err,
                           void* stream) {
  using namespace tpk;
  if (!sizes_ok(N, V, C) || !(scale > 0.f) || !(scale < INFINITY)) return TPK_E_ARG;
  if (N == 0) return TPK_OK;
  if (!h || !w || !target || !loss || !lse || !aligned16(h) || !aligned16(w)) return TPK_E_ARG;
  LmWork k;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      ws_bytes < carve(static_cast<uint8_t*>(workspace), N, V, C, false, &k))
    return TPK_E_WORKSPACE;
  int st = check_device();
  if (st != TPK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const LmShape sh = lm_shape(N, V);
  if (k.hc) st = gather_rows(h, w, target, N, V, C, k, s);
  const int32_t ld = row_stride(C);
  const float scale_log2 = scale * kLog2e;
  int slots = 2 * sh.chunks;
  if (use_few(N, C)) {
    st = few_rows(N) == 1   ? launch_few<1>(h, w, target, N, V, C, sh.np, scale_log2, &slots, k, s)
         : few_rows(N) == 2 ? launch_few<2>(h, w, target, N, V, C, sh.np, scale_log2, &slots, k, s)
                            : launch_few<4>(h, w, target, N, V, C, sh.np, scale_log2, &slots, k, s);
  } else {
    CUtensorMap ma, mb;
    if (st == TPK_OK) st = k.hc ? make_map_2d(&ma, k.hc, sh.np, C, ld, kHalf) : make_map_2d(&ma, h, N, C, C, kHalf);
    if (st == TPK_OK) st = k.wc ? make_map_2d(&mb, k.wc, V, C, ld, kHalf) : make_map_2d(&mb, w, V, C, C, kHalf);
    if (st != TPK_OK) return st;
    LmParams p{};
    p.count = k.count;
    p.n_rows = static_cast<int32_t>(N);
    p.V = static_cast<int32_t>(V);
    p.C = C;
    p.np = sh.np;
    p.rows = k.rows;
    p.target = target;
    p.scale = scale;
    p.scale_log2 = scale_log2;
    p.part = k.part;
    p.zt = k.zt;
    p.run = sh.run;
    p.err = dev_err;
    st = launch_product<kFwd>(ma, mb, ma, p, sh.np / kTile * sh.chunks, s);
  }
  if (st != TPK_OK) return st;
  const int n = static_cast<int>(N), v = static_cast<int>(V);
  if (N <= 1024)
    lm_join_kernel<4><<<(n + 3) / 4, 256, 0, s>>>(k.part, k.zt, k.pos, target, n, v, slots, sh.np, scale, scale_log2,
                                                  loss, lse);
  else
    lm_join_kernel<32><<<(n + 31) / 32, 256, 0, s>>>(k.part, k.zt, k.pos, target, n, v, slots, sh.np, scale,
                                                     scale_log2, loss, lse);
  return cuda_status(cudaGetLastError());
}

extern "C" int tpk_lm_loss_bwd(const void* h, const void* w, const int32_t* target, const float* lse,
                               const float* dloss, void* dh, void* dw, int64_t N, int64_t V, int32_t C, float scale,
                               void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream) {
  using namespace tpk;
  if (!sizes_ok(N, V, C) || !(scale > 0.f) || !(scale < INFINITY) || !dw || !aligned16(dw)) return TPK_E_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    const int st = check_device();
    return st != TPK_OK ? st : cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * C * 2, s));
  }
  if (!h || !w || !target || !lse || !dloss || !dh) return TPK_E_ARG;
  if (!aligned16(h) || !aligned16(w) || !aligned16(dh)) return TPK_E_ARG;
  LmWork k;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      ws_bytes < carve(static_cast<uint8_t*>(workspace), N, V, C, true, &k))
    return TPK_E_WORKSPACE;
  int st = check_device();
  if (st != TPK_OK) return st;
  const LmShape sh = lm_shape(N, V);
  st = gather_rows(h, w, target, N, V, C, k, s);
  const int32_t ld = row_stride(C), ldw = k.wc ? ld : C;
  const void* wt = k.wc ? k.wc : w;
  // h, w, dz: boxes of 128 rows (K-major operands, dz's and dw's way out) and of 64 (MN-major)
  CUtensorMap hk, hm, wk, wm, zk, zm, dwk;
  if (st == TPK_OK) st = make_map_2d(&hk, k.hc, sh.np, C, ld, kHalf);
  if (st == TPK_OK) st = make_map_2d(&hm, k.hc, sh.np, C, ld, 64);
  if (st == TPK_OK) st = make_map_2d(&wk, wt, V, C, ldw, kHalf);
  if (st == TPK_OK) st = make_map_2d(&wm, wt, V, C, ldw, 64);
  if (st == TPK_OK) st = make_map_2d(&zk, k.dz, sh.np, sh.piece, sh.piece, kHalf);
  if (st == TPK_OK) st = make_map_2d(&dwk, dw, V, C, C, kHalf);
  if (st == TPK_OK) st = make_map_2d(&zm, k.dz, sh.np, sh.piece, sh.piece, 64);
  LmParams p{};
  p.count = k.count;
  p.n_rows = static_cast<int32_t>(N);
  p.V = static_cast<int32_t>(V);
  p.C = C;
  p.np = sh.np;
  p.rows = k.rows;
  p.target = target;
  p.lse = lse;
  p.dloss = dloss;
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  p.ld_dz = static_cast<int32_t>(sh.piece);
  p.split_most = split_limit(static_cast<int>(((sh.piece < V ? sh.piece : V) + 63) / 64));
  p.dh = static_cast<__nv_bfloat16*>(dh);
  p.dw = static_cast<__nv_bfloat16*>(dw);
  p.err = dev_err;
  const int64_t ct = (C + kTile - 1) / kTile;
  for (int i = 0; st == TPK_OK && i < sh.pieces; ++i) {
    p.v0 = static_cast<int32_t>(i * sh.piece);
    p.vcols = static_cast<int32_t>(V - p.v0 < sh.piece ? V - p.v0 : sh.piece);
    p.first = i == 0;
    p.last = i + 1 == sh.pieces;
    const int64_t vt = (p.vcols + kTile - 1) / kTile;
    const int64_t dz_units = sh.np / kTile * vt;
    st = C <= 64 * kChunkOf<kDz> ? launch_product<kDz, true>(hk, wk, zk, p, dz_units, s)
                                 : launch_product<kDz>(hk, wk, zk, p, dz_units, s);
    if (st == TPK_OK && use_few(N, C)) {
      lm_few_target_kernel<<<1, static_cast<unsigned>(32 * N), 0, s>>>(
          static_cast<const uint4*>(h), static_cast<const uint4*>(w), target, k.pos, lse, dloss, p.v0, p.vcols, C / 8,
          scale, p.ld_dz, k.dz);
      st = cuda_status(cudaGetLastError());
    }
    p.acc = k.acc_h;
    if (st == TPK_OK) st = launch_product<kDh>(zk, wm, zk, p, INT64_MAX, s);
    p.acc = k.acc_w;
    if (st == TPK_OK)
      st = N <= 64 * kChunkOf<kDw> ? launch_product<kDw, true>(zm, hm, dwk, p, INT64_MAX, s)
                                   : launch_product<kDw>(zm, hm, dwk, p, INT64_MAX, s);
    if (st == TPK_OK && splits_for(vt * ct, split_limit(static_cast<int>(sh.np / 64))) > 1) {
      const int64_t warps = int64_t{p.vcols} * ((C / 8 + 31) / 32);
      lm_dw_kernel<<<static_cast<unsigned>(grid_for(warps)), 256, 0, s>>>(k.acc_w, k.count, p.v0, p.vcols, C,
                                                                          static_cast<uint4*>(dw));
      st = cuda_status(cudaGetLastError());
    }
  }
  if (st != TPK_OK) return st;
  lm_dh_kernel<<<static_cast<unsigned>(grid_for(N * ((C / 8 + 31) / 32))), 256, 0, s>>>(
      k.acc_h, k.pos, k.count, static_cast<int>(N), C, p.split_most, static_cast<uint4*>(dh));
  return cuda_status(cudaGetLastError());
}
