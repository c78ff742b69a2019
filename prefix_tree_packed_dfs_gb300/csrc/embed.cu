// Embedding lookup with scaling, and the table's gradient by sorted tokens.
//
// Forward: out[f] = bf16(scale * table[tokens[f]]), a zero row where the id is
// outside [0, V).  HBM-bound copy: each warp moves 128 16-byte pieces of a
// row (or of a few short rows), four per lane in flight.
//
// Backward: dtable[v] = scale * sum of dout[f] over tokens[f] = v, fp32 sums
// in ascending f (deterministic, no floating-point atomics).  The ids are
// sorted with their positions (stable radix sort, hand-written below), the
// sorted order is cut into pieces of 16 or 64 positions, and a warp adds up
// the rows of one piece for 256 columns.  A run of equal ids inside a piece is
// written straight to its row of dtable; a run that crosses pieces leaves one
// fp32 partial per piece, and a second kernel adds those in order -- so a
// frequent id (thousands of rows) is spread over as many warps as it has
// pieces.  Rows of ids that do not occur are zeroed: the highest ids by other
// CTAs of the sort's launches, which leave the memory idle, the rest by other
// CTAs of the sums' launch, which look the id up in the sorted order (32-way
// search, so those rows are written once).
// Measured on GB300, 96,888 rows of 2,048, 32,000 ids: lookup from an fp32
// table 106 us (6.2 TB/s of the least bytes), from a bf16 one 80 us (6.6);
// gradient 141 us, of which the sums are HBM-bound.  Rows cleared under the
// sort, 48 MB per launch: 143 -> 141 us here, 60 -> 55 for 30,000 rows of
// 1,024 into 30,000 (24 MB 56, 80 MB 61: then the sort waits for the memory).
// 1,001 rows of 1,000: 11 us, three launches.
#include <type_traits>

#include "rowwise.cuh"

namespace tpk {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 scale8(uint4 x, float s) {
  return make_uint4(pack2(lo16(x.x) * s, hi16(x.x) * s), pack2(lo16(x.y) * s, hi16(x.y) * s),
                    pack2(lo16(x.z) * s, hi16(x.z) * s), pack2(lo16(x.w) * s, hi16(x.w) * s));
}

// ---- forward ---------------------------------------------------------------
// lanes_log2: lanes that share a row (a row of C/8 16-byte outputs); a warp
// item is (32 >> lanes_log2 rows) x (4 << lanes_log2 outputs of each).
template <bool kF32>
__global__ void __launch_bounds__(kThreads) embed_kernel(const void* __restrict__ table,
                                                         const int32_t* __restrict__ tokens, int64_t N, int64_t V,
                                                         uint4* __restrict__ out, int vecs, int lanes_log2, int parts,
                                                         float scale) {
  const int lane = threadIdx.x & 31;
  const int rows_per = 32 >> lanes_log2;
  const int64_t items = ((N + rows_per - 1) / rows_per) * parts;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += warps) {
    const int64_t f = it / parts * rows_per + (lane >> lanes_log2);
    if (f >= N) continue;
    const int c0 = static_cast<int>(it % parts) * (4 << lanes_log2) + (lane & ((1 << lanes_log2) - 1));
    const int tok = __ldg(tokens + f);
    const bool in = tok >= 0 && tok < V;
    uint4 r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + (j << lanes_log2);
      r[j] = make_uint4(0, 0, 0, 0);
      if (in && c < vecs) {
        if constexpr (kF32) {
          const float4* src = static_cast<const float4*>(table) + (static_cast<int64_t>(tok) * vecs + c) * 2;
          const float4 a = __ldg(src), b = __ldg(src + 1);
          r[j] = make_uint4(pack2(a.x * scale, a.y * scale), pack2(a.z * scale, a.w * scale),
                            pack2(b.x * scale, b.y * scale), pack2(b.z * scale, b.w * scale));
        } else {
          r[j] = __ldg(static_cast<const uint4*>(table) + static_cast<int64_t>(tok) * vecs + c);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + (j << lanes_log2);
      if (c < vecs) out[f * vecs + c] = kF32 || !in ? r[j] : scale8(r[j], scale);
    }
  }
}

// ---- backward: stable radix sort of (id, position) ---------------------------
// Tiles of kSortThreads * kRounds consecutive positions, one CTA each; a digit
// has 8 bits.  A warp holds its contiguous run of the tile in registers, 32
// keys per round, and ranks a key among the warp's earlier keys of the same
// digit (__match_any_sync and a per-warp count per digit).
// One tile (N <= 2048): one CTA runs every pass in shared memory.  More: the
// first pass's counts hist[tile][digit] come from sort_hist_kernel; every
// scatter pass counts the next digit of the tile each key lands in (integer
// atomics: the counts do not depend on their order), and a scatter CTA adds
// up the counts of all tiles itself, which costs tiles * 1 KB of L2 reads and
// saves a scan launch.
constexpr int kDigits = 256;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kFewRounds = 4, kManyRounds = 16;
constexpr int64_t kFewTiles = 512;   // up to here tiles of kFewRounds

// The sort leaves the memory idle, so its launches carry CTAs that clear rows
// of dtable meanwhile: the highest ids, kClear bytes per launch (what the
// memory writes in a pass's time); rows whose ids do occur are written later.
constexpr int64_t kClear = int64_t{48} << 20;
struct Clear {
  uint4* at;     // the launch's rows, 16-byte pieces
  int64_t n;
};
__device__ __forceinline__ void clear_rows(const Clear& z, int block, int blocks) {
  for (int64_t i = static_cast<int64_t>(block) * kSortThreads + threadIdx.x; i < z.n;
       i += static_cast<int64_t>(blocks) * kSortThreads)
    z.at[i] = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ int key_of(int tok, int V) { return tok >= 0 && tok < V ? tok : V; }

// Inclusive scan of one value per thread over the first 256 threads (8 warps);
// every thread of the CTA calls it.
__device__ __forceinline__ int scan256(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (warp < 8 && lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp < 8)
    for (int w = 0; w < warp; ++w) v += warp_sums[w];
  return v;
}

// The warp's keys' ranks among its keys of the same digit; count[d] (the
// warp's, zeroed) receives how many there are of each.
template <int kRounds>
__device__ __forceinline__ void rank_keys(const int (&key)[kRounds], int n, int shift, int* count,
                                          int (&rank)[kRounds]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const bool in = r * 32 + lane < n;
    const int d = in ? (key[r] >> shift) & (kDigits - 1) : kDigits;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const int before = in ? count[d] : 0;
    rank[r] = before + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (in && lane == __ffs(same) - 1) count[d] = before + __popc(same);
    __syncwarp();
  }
}

template <int kRounds>
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(const int32_t* __restrict__ tokens, int N, int V,
                                                                 int passes, int32_t* __restrict__ hist) {
  __shared__ int h[kDigits];
  const int tiles = gridDim.x, tile = blockIdx.x;
  const int64_t lo = static_cast<int64_t>(tile) * (kSortThreads * kRounds);
  int key[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = lo + r * kSortThreads + threadIdx.x;
    key[r] = i < N ? key_of(__ldg(tokens + i), V) : -1;
  }
  if (threadIdx.x < kDigits) {
    h[threadIdx.x] = 0;
    for (int p = 1; p < passes; ++p) hist[(static_cast<int64_t>(p) * tiles + tile) * kDigits + threadIdx.x] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (key[r] >= 0) atomicAdd(&h[key[r] & (kDigits - 1)], 1);
  __syncthreads();
  if (threadIdx.x < kDigits) hist[static_cast<int64_t>(tile) * kDigits + threadIdx.x] = h[threadIdx.x];
}

// One pass: keys_in (nullptr: the ids themselves, positions 0..N-1) sorted by
// the 8 bits at `shift`.
template <int kRounds>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const int32_t* __restrict__ tokens,
                                                                    const int32_t* __restrict__ keys_in,
                                                                    const int32_t* __restrict__ pos_in, int N, int V,
                                                                    int shift, const int32_t* __restrict__ hist,
                                                                    int32_t* __restrict__ hist_next,
                                                                    int32_t* __restrict__ keys_out,
                                                                    int32_t* __restrict__ pos_out, int tiles,
                                                                    Clear clear) {
  if (static_cast<int>(blockIdx.x) >= tiles) return clear_rows(clear, blockIdx.x - tiles, gridDim.x - tiles);
  __shared__ int base[kSortWarps][kDigits];   // counts, then where each warp's keys of a digit go
  __shared__ int warp_sums[8];
  constexpr int kPer = kSortThreads * kRounds, kRun = 32 * kRounds;
  const int tile = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t lo = static_cast<int64_t>(tile) * kPer + warp * kRun;
  const int n = lo >= N ? 0 : static_cast<int>(N - lo < kRun ? N - lo : kRun);   // the warp's keys
  int key[kRounds], pos[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = lo + r * 32 + lane;
    const bool in = r * 32 + lane < n;
    key[r] = !in ? 0 : keys_in ? __ldg(keys_in + i) : key_of(__ldg(tokens + i), V);
    pos[r] = !in ? 0 : pos_in ? __ldg(pos_in + i) : static_cast<int>(i);
  }
  int before = 0, total = 0;   // this digit's keys in earlier tiles, in all tiles
  if (threadIdx.x < kDigits) {
    const int32_t* hd = hist + threadIdx.x;
#pragma unroll 16
    for (int t = 0; t < tiles; ++t) {
      const int c = __ldg(hd + static_cast<int64_t>(t) * kDigits);
      total += c;
      before += t < tile ? c : 0;
    }
  }
  for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads) (&base[0][0])[i] = 0;
  __syncthreads();
  rank_keys<kRounds>(key, n, shift, base[warp], rank);
  int at = scan256(total, warp_sums) - total + before;   // its barrier also ends the ranking
  if (threadIdx.x < kDigits) {
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = base[w][threadIdx.x];
      base[w][threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (r * 32 + lane >= n) continue;
    const int to = base[warp][(key[r] >> shift) & (kDigits - 1)] + rank[r];
    keys_out[to] = key[r];
    pos_out[to] = pos[r];
    if (hist_next)
      atomicAdd(hist_next + static_cast<int64_t>(to / kPer) * kDigits + ((key[r] >> (shift + 8)) & (kDigits - 1)), 1);
  }
}

// Every pass of a single tile, in shared memory.
__global__ void __launch_bounds__(kSortThreads) sort_one_kernel(const int32_t* __restrict__ tokens, int N, int V,
                                                                int passes, int32_t* __restrict__ keys_out,
                                                                int32_t* __restrict__ pos_out, Clear clear) {
  if (blockIdx.x > 0) return clear_rows(clear, blockIdx.x - 1, gridDim.x - 1);
  constexpr int kPer = kSortThreads * kFewRounds, kRun = 32 * kFewRounds;
  __shared__ int base[kSortWarps][kDigits];
  __shared__ int warp_sums[8];
  __shared__ int sk[kPer], sp[kPer];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lo = warp * kRun;
  const int n = lo >= N ? 0 : min(N - lo, kRun);
  int key[kFewRounds], pos[kFewRounds], rank[kFewRounds];
#pragma unroll
  for (int r = 0; r < kFewRounds; ++r) {
    pos[r] = lo + r * 32 + lane;
    key[r] = r * 32 + lane < n ? key_of(__ldg(tokens + pos[r]), V) : 0;
  }
  for (int p = 0; p < passes; ++p) {
    for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads) (&base[0][0])[i] = 0;
    __syncthreads();
    rank_keys<kFewRounds>(key, n, 8 * p, base[warp], rank);
    __syncthreads();
    int total = 0;
    if (threadIdx.x < kDigits)
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) total += base[w][threadIdx.x];
    int at = scan256(total, warp_sums) - total;
    if (threadIdx.x < kDigits) {
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = base[w][threadIdx.x];
        base[w][threadIdx.x] = at;
        at += c;
      }
    }
    __syncthreads();
    const bool last = p + 1 == passes;
#pragma unroll
    for (int r = 0; r < kFewRounds; ++r) {
      if (r * 32 + lane >= n) continue;
      const int to = base[warp][(key[r] >> (8 * p)) & (kDigits - 1)] + rank[r];
      (last ? keys_out : sk)[to] = key[r];
      (last ? pos_out : sp)[to] = pos[r];
    }
    if (last) return;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kFewRounds; ++r) {
      const int i = lo + r * 32 + lane;
      if (r * 32 + lane < n) {
        key[r] = sk[i];
        pos[r] = sp[i];
      }
    }
    __syncthreads();
  }
}

// ---- backward: sums of runs ---------------------------------------------------
constexpr int kCols = 256;        // columns per warp (8 per lane)
constexpr int kBatch = 8;         // rows loaded together

// Sorted positions per piece: long pieces leave fewer partials, short ones
// give a small batch more warps (1,001 rows of 1,000: 16 beats 64).
__host__ __device__ constexpr int piece_for(int64_t N) { return N >= 16384 ? 64 : 16; }

template <bool kF32>
__device__ __forceinline__ void store_row8(void* dst, int64_t at, const float (&a)[8], float s) {
  if constexpr (kF32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(dst) + at);
    d[0] = make_float4(a[0] * s, a[1] * s, a[2] * s, a[3] * s);
    d[1] = make_float4(a[4] * s, a[5] * s, a[6] * s, a[7] * s);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + at) =
        make_uint4(pack2(a[0] * s, a[1] * s), pack2(a[2] * s, a[3] * s), pack2(a[4] * s, a[5] * s),
                   pack2(a[6] * s, a[7] * s));
  }
}

// First index of the ascending keys[0, n) that is >= key: 32-way search by a warp.
__device__ __forceinline__ int lower_bound_warp(const int32_t* __restrict__ keys, int n, int key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;   // the answer lies in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const bool less = i < lo + len && __ldg(keys + i) < key;
    const int k = __popc(__ballot_sync(0xffffffffu, less));   // probes 0..k-1 are less
    if (k == 0) return lo;
    const int nlo = lo + (k - 1) * step + 1;
    len = min(step - 1, lo + len - nlo);
    lo = nlo;
  }
  return lo;
}

// Partials: part[(2 * piece + side) * C]: side 0 the piece's first run where
// it began in an earlier piece, side 1 its last run where it goes on in a
// later one (a piece that is all one run with both neighbours uses side 0).
template <bool kF32, int kPiece>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const int32_t* __restrict__ keys,
                                                             const int32_t* __restrict__ pos,
                                                             const uint4* __restrict__ dout, int N, int V, int C,
                                                             float scale, void* __restrict__ dtable,
                                                             float* __restrict__ part, int sum_blocks, int cleared) {
  const int lane = threadIdx.x & 31;
  const int parts = (C + kCols - 1) / kCols;
  if (static_cast<int>(blockIdx.x) >= sum_blocks) {
    // rows of ids that do not occur, up to those cleared under the sort
    const int64_t warps = static_cast<int64_t>(gridDim.x - sum_blocks) * (kThreads / 32);
    for (int64_t v = static_cast<int64_t>(blockIdx.x - sum_blocks) * (kThreads / 32) + (threadIdx.x >> 5);
         v < cleared; v += warps) {
      const int i = lower_bound_warp(keys, N, static_cast<int>(v));
      if (i < N && __ldg(keys + i) == v) continue;
      const int n16 = C * (kF32 ? 4 : 2) / 16;
      uint4* d = static_cast<uint4*>(dtable) + v * n16;
      for (int c = lane; c < n16; c += 32) d[c] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t piece = item / parts;
  const int c = static_cast<int>(item % parts) * kCols + lane * 8;
  const int64_t lo = piece * kPiece;
  if (lo >= N) return;
  const int n = static_cast<int>(N - lo < kPiece ? N - lo : kPiece);
  const int vecs = C / 8;
  const bool col = c < C;
  // the piece's ids and positions, one per lane and 32 of them
  constexpr int kHeld = (kPiece + 31) / 32;
  int hk[kHeld], hp[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int e = i * 32 + lane;
    hk[i] = e < n ? __ldg(keys + lo + e) : -2;
    hp[i] = e < n ? __ldg(pos + lo + e) : 0;
  }
  const int prev = lo > 0 ? __ldg(keys + lo - 1) : -1;
  const int next = lo + n < N ? __ldg(keys + lo + n) : -1;
  uint4 x[2][kBatch];
  auto fetch = [&](int b, uint4 (&to)[kBatch]) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int e = b + j;   // a constant once unrolled
      const int k = __shfl_sync(0xffffffffu, hk[e / 32], e % 32), q = __shfl_sync(0xffffffffu, hp[e / 32], e % 32);
      to[j] = make_uint4(0, 0, 0, 0);
      if (k >= 0 && k < V && col) to[j] = __ldg(dout + static_cast<int64_t>(q) * vecs + c / 8);
    }
  };
  float acc[8] = {};
  int cur = __shfl_sync(0xffffffffu, hk[0], 0);
  bool joined = cur == prev;   // the current run began in an earlier piece
  fetch(0, x[0]);
#pragma unroll
  for (int b = 0; b < kPiece; b += kBatch) {
    uint4(&now)[kBatch] = x[(b / kBatch) & 1];
    if (b + kBatch < kPiece) fetch(b + kBatch, x[(b / kBatch + 1) & 1]);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int e = b + j;
      const int k = __shfl_sync(0xffffffffu, hk[e / 32], e % 32);
      if (e < n && k != cur) {   // the run `cur` ends here
        if (col && cur < V) {
          if (joined)
            store_row8<true>(part, (2 * piece) * C + c, acc, 1.f);
          else
            store_row8<kF32>(dtable, static_cast<int64_t>(cur) * C + c, acc, scale);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        cur = k;
        joined = false;
      }
      acc[0] += lo16(now[j].x); acc[1] += hi16(now[j].x);
      acc[2] += lo16(now[j].y); acc[3] += hi16(now[j].y);
      acc[4] += lo16(now[j].z); acc[5] += hi16(now[j].z);
      acc[6] += lo16(now[j].w); acc[7] += hi16(now[j].w);
    }
  }
  if (col && cur < V) {
    if (joined)
      store_row8<true>(part, (2 * piece) * C + c, acc, 1.f);
    else if (cur == next)
      store_row8<true>(part, (2 * piece + 1) * C + c, acc, 1.f);
    else
      store_row8<kF32>(dtable, static_cast<int64_t>(cur) * C + c, acc, scale);
  }
}

// A run that crosses pieces: a warp of its first piece adds side 1 of that
// piece and side 0 of the following ones, in order, for 128 columns.  A run
// of thousands of positions is hundreds of dependent additions, so what
// counts is the loads in flight: 16 pieces at a time (4 first: most runs are
// short), whether or not they still belong to the run -- a piece does if it
// begins with the run's id, and those ids arrive with the partials.
template <bool kF32, int kPiece>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const int32_t* __restrict__ keys, int N, int V, int C,
                                                              float scale, void* __restrict__ dtable,
                                                              const float* __restrict__ part) {
  const int lane = threadIdx.x & 31;
  const int parts = (C + 127) / 128;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t piece = item / parts;
  const int c = static_cast<int>(item % parts) * 128 + lane * 4;
  const int64_t lo = piece * kPiece, hi = lo + kPiece;
  if (hi >= N) return;
  const int64_t pieces = (static_cast<int64_t>(N) + kPiece - 1) / kPiece;
  const int key = __ldg(keys + hi - 1), next = __ldg(keys + hi);
  const int begin = __ldg(keys + lo), prev = lo > 0 ? __ldg(keys + lo - 1) : -1;
  if (key >= V || next != key) return;
  if (begin == key && prev == key) return;   // the run began earlier: an earlier piece adds it up
  const bool col = c < C;
  const float* from = part + (col ? c : 0);
  float4 acc = __ldcg(reinterpret_cast<const float4*>(from + (2 * piece + 1) * C));
  // the pieces p .. p + kBatchOf - 1; false once one of them is past the run
  auto add = [&](int64_t p, auto batch) {
    constexpr int kBatchOf = decltype(batch)::value;
    const int first = lane < kBatchOf && p + lane < pieces ? __ldg(keys + (p + lane) * kPiece) : -1;
    float4 v[kBatchOf];
    auto at = [&](int i) { return from + 2 * (p + i < pieces ? p + i : pieces - 1) * C; };
    int last = 0;
#pragma unroll
    for (int i = 0; i < kBatchOf; ++i) {
      v[i] = __ldcg(reinterpret_cast<const float4*>(at(i)));
      last ^= __float_as_int(v[i].w);
    }
    // how many of them belong: sorted, so the first n.  n is made to depend on
    // every load (each lane's own value, shuffled to itself, cancels), or the
    // compiler would issue each load behind the addition of the one before.
    const int n = __popc(__ballot_sync(0xffffffffu, first == key)) ^ last ^ __shfl_sync(0xffffffffu, last, lane);
#pragma unroll
    for (int i = 0; i < kBatchOf; ++i)
      if (i < n) {
        acc.x += v[i].x; acc.y += v[i].y; acc.z += v[i].z; acc.w += v[i].w;
      }
    return n == kBatchOf;
  };
  int64_t p = piece + 1;
  if (add(p, std::integral_constant<int, 4>{}))
    for (p += 4; add(p, std::integral_constant<int, 16>{}); p += 16) {
    }
  if (!col) return;
  const int64_t at = static_cast<int64_t>(key) * C + c;
  if constexpr (kF32)
    *reinterpret_cast<float4*>(static_cast<float*>(dtable) + at) =
        make_float4(acc.x * scale, acc.y * scale, acc.z * scale, acc.w * scale);
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dtable) + at) =
        make_uint2(pack2(acc.x * scale, acc.y * scale), pack2(acc.z * scale, acc.w * scale));
}

// ---- host ------------------------------------------------------------------------
struct SortShape {
  int passes, rounds;
  int64_t tiles;
};
SortShape sort_shape(int64_t N, int64_t V) {
  SortShape s;
  s.passes = 1;
  while (s.passes < 4 && (V >> (8 * s.passes)) != 0) ++s.passes;   // keys 0..V
  s.rounds = N <= kFewTiles * kSortThreads * kFewRounds ? kFewRounds : kManyRounds;
  const int64_t per = int64_t{kSortThreads} * s.rounds;
  s.tiles = (N + per - 1) / per;
  return s;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The rows of dtable still to be cleared, [0, rows): the sort's launches take
// from the end.
struct Clearing {
  uint8_t* dtable;
  int64_t rows, row_bytes;
  Clear next() {
    int64_t n = kClear / row_bytes;
    n = n < rows ? n : rows;
    rows -= n;
    return {reinterpret_cast<uint4*>(dtable + rows * row_bytes), n * row_bytes / 16};
  }
};
unsigned clear_blocks(const Clear& c) {
  const int64_t want = (c.n + 4 * kSortThreads - 1) / (4 * kSortThreads), most = int64_t{num_sms()} * 2;
  return static_cast<unsigned>(want < most ? want : most);
}

template <int kRounds>
int sort_tiles(const int32_t* tokens, int n, int v, const SortShape& sh, int32_t* hist, int32_t* const (&buf)[4],
               Clearing* z, const int32_t** keys, const int32_t** pos, cudaStream_t s) {
  const unsigned tiles = static_cast<unsigned>(sh.tiles);
  sort_hist_kernel<kRounds><<<tiles, kSortThreads, 0, s>>>(tokens, n, v, sh.passes, hist);
  int st = cuda_status(cudaGetLastError());
  const int32_t *ki = nullptr, *pi = nullptr;
  for (int p = 0; st == TPK_OK && p < sh.passes; ++p) {
    int32_t* ko = buf[(p & 1) * 2];
    int32_t* po = buf[(p & 1) * 2 + 1];
    int32_t* h = hist + static_cast<int64_t>(p) * sh.tiles * kDigits;
    const Clear c = z->next();
    sort_scatter_kernel<kRounds><<<tiles + clear_blocks(c), kSortThreads, 0, s>>>(
        tokens, ki, pi, n, v, 8 * p, h, p + 1 < sh.passes ? h + sh.tiles * kDigits : nullptr, ko, po,
        static_cast<int>(tiles), c);
    st = cuda_status(cudaGetLastError());
    ki = ko;
    pi = po;
  }
  *keys = ki;
  *pos = pi;
  return st;
}

template <bool kF32, int kPiece>
int sum_runs(const int32_t* keys, const int32_t* pos, const void* dout, int n, int v, int C, float scale, void* dtable,
             float* part, int cleared, cudaStream_t s) {
  const int64_t pieces = (static_cast<int64_t>(n) + kPiece - 1) / kPiece;
  const int64_t sum_blocks = (pieces * ((C + kCols - 1) / kCols) + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t join_blocks = (pieces * ((C + 127) / 128) + kThreads / 32 - 1) / (kThreads / 32);
  int64_t zero_blocks = (static_cast<int64_t>(cleared) + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = int64_t{num_sms()} * 8;
  if (zero_blocks > most) zero_blocks = most;
  if (sum_blocks + zero_blocks > 0x7fffffff || join_blocks > 0x7fffffff) return TPK_E_ARG;
  embed_sum_kernel<kF32, kPiece><<<static_cast<unsigned>(sum_blocks + zero_blocks), kThreads, 0, s>>>(
      keys, pos, static_cast<const uint4*>(dout), n, v, C, scale, dtable, part, static_cast<int>(sum_blocks),
      cleared);
  const int st = cuda_status(cudaGetLastError());
  if (st != TPK_OK || pieces < 2) return st;
  embed_join_kernel<kF32, kPiece><<<static_cast<unsigned>(join_blocks), kThreads, 0, s>>>(keys, n, v, C, scale, dtable,
                                                                                          part);
  return cuda_status(cudaGetLastError());
}

bool sizes_ok(int64_t N, int64_t V, int32_t C) {
  return N >= 0 && N < (int64_t{1} << 31) - 8192 && V >= 1 && V < (int64_t{1} << 31) - 1 && C >= 8 && C % 8 == 0 &&
         C <= (1 << 20);
}

}  // namespace
}  // namespace tpk

extern "C" int tpk_embed(const void* table, int32_t table_type, const int32_t* tokens, void* out, int64_t N, int64_t V,
                         int32_t C, float scale, void* stream) {
  using namespace tpk;
  if (!sizes_ok(N, V, C) || (table_type != TPK_BF16 && table_type != TPK_F32)) return TPK_E_ARG;
  if (N == 0) return TPK_OK;
  if (!table || !tokens || !out) return TPK_E_ARG;
  if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(out)) % 16) return TPK_E_ARG;
  int st = check_device();
  if (st != TPK_OK) return st;
  const int vecs = C / 8;
  const int ll = vecs <= 8 ? 3 : vecs <= 16 ? 4 : 5;
  const int parts = (vecs + (4 << ll) - 1) / (4 << ll);
  const int rows_per = 32 >> ll;
  const int64_t items = (N + rows_per - 1) / rows_per * parts;
  int64_t blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = int64_t{num_sms()} * 16;
  if (blocks > most) blocks = most;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (table_type == TPK_F32)
    embed_kernel<true><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(table, tokens, N, V, static_cast<uint4*>(out),
                                                                          vecs, ll, parts, scale);
  else
    embed_kernel<false><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(table, tokens, N, V,
                                                                           static_cast<uint4*>(out), vecs, ll, parts,
                                                                           scale);
  return cuda_status(cudaGetLastError());
}

extern "C" size_t tpk_embed_bwd_workspace_bytes(int64_t N, int64_t V, int32_t C) {
  using namespace tpk;
  if (!sizes_ok(N, V, C)) return 0;
  const SortShape s = sort_shape(N, V);
  const size_t n = static_cast<size_t>(N);
  const size_t piece = static_cast<size_t>(piece_for(N));
  const size_t pieces = (n + piece - 1) / piece;
  return up256(static_cast<size_t>(s.passes) * s.tiles * kDigits * 4) + 4 * up256(n * 4) +
         up256(pieces * 2 * static_cast<size_t>(C) * 4);
}

extern "C" int tpk_embed_bwd(const int32_t* tokens, const void* dout, void* dtable, int32_t table_type, int64_t N,
                             int64_t V, int32_t C, float scale, void* workspace, size_t ws_bytes, void* stream) {
  using namespace tpk;
  if (!sizes_ok(N, V, C) || (table_type != TPK_BF16 && table_type != TPK_F32) || !dtable) return TPK_E_ARG;
  if (N > 0 && (!tokens || !dout)) return TPK_E_ARG;
  if ((reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(dtable)) % 16) return TPK_E_ARG;
  const size_t need = tpk_embed_bwd_workspace_bytes(N, V, C);
  if (N > 0 && (!workspace || ws_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256)) return TPK_E_WORKSPACE;
  int st = check_device();
  if (st != TPK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = table_type == TPK_F32;
  if (N == 0)
    return cuda_status(cudaMemsetAsync(dtable, 0, static_cast<size_t>(V) * C * (f32 ? 4 : 2), s));
  const SortShape sh = sort_shape(N, V);
  const int n = static_cast<int>(N), v = static_cast<int>(V);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  int32_t* hist = reinterpret_cast<int32_t*>(w);
  w += up256(static_cast<size_t>(sh.passes) * sh.tiles * kDigits * 4);
  int32_t* buf[4];
  for (auto& b : buf) {
    b = reinterpret_cast<int32_t*>(w);
    w += up256(static_cast<size_t>(N) * 4);
  }
  float* part = reinterpret_cast<float*>(w);
  const int32_t *ki = buf[0], *pi = buf[1];
  Clearing z{static_cast<uint8_t*>(dtable), V, int64_t{C} * (f32 ? 4 : 2)};
  if (sh.tiles == 1) {
    const Clear c = z.next();
    sort_one_kernel<<<1 + clear_blocks(c), kSortThreads, 0, s>>>(tokens, n, v, sh.passes, buf[0], buf[1], c);
    st = cuda_status(cudaGetLastError());
  } else {
    st = sh.rounds == kFewRounds ? sort_tiles<kFewRounds>(tokens, n, v, sh, hist, buf, &z, &ki, &pi, s)
                                 : sort_tiles<kManyRounds>(tokens, n, v, sh, hist, buf, &z, &ki, &pi, s);
  }
  if (st != TPK_OK) return st;
  const bool few = piece_for(N) == 16;
  const int left = static_cast<int>(z.rows);
  if (f32)
    return few ? sum_runs<true, 16>(ki, pi, dout, n, v, C, scale, dtable, part, left, s)
               : sum_runs<true, 64>(ki, pi, dout, n, v, C, scale, dtable, part, left, s);
  return few ? sum_runs<false, 16>(ki, pi, dout, n, v, C, scale, dtable, part, left, s)
             : sum_runs<false, 64>(ki, pi, dout, n, v, C, scale, dtable, part, left, s);
}
