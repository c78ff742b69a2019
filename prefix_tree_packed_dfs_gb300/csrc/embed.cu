// Embedding lookup with scaling, and the table's gradient by sorted tokens.
//
// Forward: out[f] = bf16(scale * table[tokens[f]]), a zero row where the id is
// outside [0, V).  HBM-bound copy: each warp moves 128 16-byte pieces of a
// row (or of a few short rows), four per lane in flight.
//
// Backward: dtable[v] = scale * sum of dout[f] over tokens[f] = v, fp32 sums
// in ascending f (deterministic, no floating-point atomics).  The ids are
// sorted with their positions (stable radix sort, hand-written below), the
// sorted order is cut into pieces of kPiece positions, and a warp adds up the
// rows of one piece for 256 columns.  A run of equal ids inside a piece is
// written straight to its row of dtable; a run that crosses pieces leaves one
// fp32 partial per piece, and a second kernel adds those in order -- so a
// frequent id (thousands of rows) is spread over as many warps as it has
// pieces.  Rows of ids that do not occur are zeroed by other blocks of the
// same launch, which look the id up in the sorted order (32-way search, so
// the table is written once instead of cleared and written again).
#include <cuda_bf16.h>

#include "common.cuh"

namespace tpk {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

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
// Tiles of `per` consecutive positions, one CTA each; a digit has 8 bits.
// hist[pass][tile][digit] counts the tile's keys.  The first pass's counts
// come from sort_hist_kernel; every scatter pass counts the next digit of the
// tile each key lands in (integer atomics: the counts do not depend on their
// order).  A scatter CTA adds up the counts of all tiles itself, which costs
// tiles * 1 KB of L2 reads and saves a scan launch.
constexpr int kDigits = 256;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMinTile = 2048;
constexpr int kMaxTiles = 512;

__device__ __forceinline__ int key_of(int tok, int V) { return tok >= 0 && tok < V ? tok : V; }

__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(const int32_t* __restrict__ tokens, int N, int V,
                                                                 int per, int passes, int32_t* __restrict__ hist) {
  __shared__ int h[kDigits];
  const int tiles = gridDim.x, tile = blockIdx.x;
  if (threadIdx.x < kDigits) h[threadIdx.x] = 0;
  __syncthreads();
  const int lo = tile * per, hi = min(N, lo + per);
  for (int i = lo + threadIdx.x; i < hi; i += kSortThreads) atomicAdd(&h[key_of(__ldg(tokens + i), V) & (kDigits - 1)], 1);
  __syncthreads();
  if (threadIdx.x < kDigits) {
    hist[tile * kDigits + threadIdx.x] = h[threadIdx.x];
    for (int p = 1; p < passes; ++p) hist[(p * tiles + tile) * kDigits + threadIdx.x] = 0;
  }
}

// One pass: keys_in (nullptr: the ids themselves, positions 0..N-1) sorted by
// the 8 bits at `shift`.  per is a multiple of 32 * kSortWarps; a warp ranks
// its own contiguous run of the tile, 32 keys at a time.
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const int32_t* __restrict__ tokens,
                                                                    const int32_t* __restrict__ keys_in,
                                                                    const int32_t* __restrict__ pos_in, int N, int V,
                                                                    int per, int shift, const int32_t* __restrict__ hist,
                                                                    int32_t* __restrict__ hist_next,
                                                                    int32_t* __restrict__ keys_out,
                                                                    int32_t* __restrict__ pos_out) {
  __shared__ int base[kSortWarps][kDigits];   // counts, then where each warp's keys of a digit go
  __shared__ int scan[kDigits];
  const int tiles = gridDim.x, tile = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads) (&base[0][0])[i] = 0;
  __syncthreads();
  const int run = per / kSortWarps;
  const int lo = tile * per + warp * run, hi = min(N, min(tile * per + per, lo + run));
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const int key = i < hi ? (keys_in ? __ldg(keys_in + i) : key_of(__ldg(tokens + i), V)) : 0;
    const int d = i < hi ? (key >> shift) & (kDigits - 1) : kDigits;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    if (i < hi && lane == __ffs(same) - 1) base[warp][d] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  int before = 0, total = 0;   // this digit's keys in earlier tiles, in all tiles
  if (threadIdx.x < kDigits) {
    const int32_t* hd = hist + threadIdx.x;
#pragma unroll 8
    for (int t = 0; t < tiles; ++t) {
      const int c = __ldg(hd + t * kDigits);
      total += c;
      before += t < tile ? c : 0;
    }
    scan[threadIdx.x] = total;
  }
  __syncthreads();
  for (int o = 1; o < kDigits; o <<= 1) {
    const int add = threadIdx.x < kDigits && threadIdx.x >= o ? scan[threadIdx.x - o] : 0;
    __syncthreads();
    if (threadIdx.x < kDigits) scan[threadIdx.x] += add;
    __syncthreads();
  }
  if (threadIdx.x < kDigits) {
    int at = scan[threadIdx.x] - total + before;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = base[w][threadIdx.x];
      base[w][threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < hi;
    const int key = in ? (keys_in ? __ldg(keys_in + i) : key_of(__ldg(tokens + i), V)) : 0;
    const int d = in ? (key >> shift) & (kDigits - 1) : kDigits;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    int to = 0;
    if (in) to = base[warp][d] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (in && lane == __ffs(same) - 1) base[warp][d] += __popc(same);
    __syncwarp();
    if (in) {
      keys_out[to] = key;
      pos_out[to] = pos_in ? __ldg(pos_in + i) : i;
      if (hist_next) atomicAdd(hist_next + (to / per) * kDigits + ((key >> (shift + 8)) & (kDigits - 1)), 1);
    }
  }
}

// ---- backward: sums of runs ---------------------------------------------------
constexpr int kPiece = 64;        // sorted positions per piece
constexpr int kCols = 256;        // columns per warp (8 per lane)
constexpr int kAhead = 8;         // rows in flight per warp

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
template <bool kF32>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const int32_t* __restrict__ keys,
                                                             const int32_t* __restrict__ pos,
                                                             const uint4* __restrict__ dout, int N, int V, int C,
                                                             float scale, void* __restrict__ dtable,
                                                             float* __restrict__ part, int sum_blocks) {
  const int lane = threadIdx.x & 31;
  const int parts = (C + kCols - 1) / kCols;
  if (static_cast<int>(blockIdx.x) >= sum_blocks) {
    // rows of ids that do not occur
    const int64_t warps = static_cast<int64_t>(gridDim.x - sum_blocks) * (kThreads / 32);
    for (int64_t v = static_cast<int64_t>(blockIdx.x - sum_blocks) * (kThreads / 32) + (threadIdx.x >> 5); v < V;
         v += warps) {
      const int i = lower_bound_warp(keys, N, static_cast<int>(v));
      if (i < N && __ldg(keys + i) == v) continue;
      const int n16 = C * (kF32 ? 4 : 2) / 16;
      uint4* d = static_cast<uint4*>(dtable) + v * n16;
      for (int c = lane; c < n16; c += 32) d[c] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int piece = static_cast<int>(item / parts);
  const int c = static_cast<int>(item % parts) * kCols + lane * 8;
  const int lo = piece * kPiece;
  if (lo >= N) return;
  const int hi = min(N, lo + kPiece);
  const int vecs = C / 8;
  const bool col = c < C;
  const int prev = lo > 0 ? __ldg(keys + lo - 1) : -1;
  const int next = hi < N ? __ldg(keys + hi) : -1;
  float acc[8] = {};
  int cur = __ldg(keys + lo);
  bool joined = cur == prev;   // the current run began in an earlier piece
  for (int b = lo; b < hi; b += kAhead) {
    uint4 x[kAhead];
    int k[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      k[j] = b + j < hi ? __ldg(keys + b + j) : -2;
      x[j] = make_uint4(0, 0, 0, 0);
      if (b + j < hi && k[j] < V && col) x[j] = __ldg(dout + static_cast<int64_t>(__ldg(pos + b + j)) * vecs + c / 8);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (b + j >= hi) break;
      if (k[j] != cur) {   // the run `cur` ends here
        if (col && cur < V) {
          if (joined)
            store_row8<true>(part, (2ll * piece) * C + c, acc, 1.f);
          else
            store_row8<kF32>(dtable, static_cast<int64_t>(cur) * C + c, acc, scale);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        cur = k[j];
        joined = false;
      }
      acc[0] += lo16(x[j].x); acc[1] += hi16(x[j].x);
      acc[2] += lo16(x[j].y); acc[3] += hi16(x[j].y);
      acc[4] += lo16(x[j].z); acc[5] += hi16(x[j].z);
      acc[6] += lo16(x[j].w); acc[7] += hi16(x[j].w);
    }
  }
  if (col && cur < V) {
    if (joined)
      store_row8<true>(part, (2ll * piece) * C + c, acc, 1.f);
    else if (cur == next)
      store_row8<true>(part, (2ll * piece + 1) * C + c, acc, 1.f);
    else
      store_row8<kF32>(dtable, static_cast<int64_t>(cur) * C + c, acc, scale);
  }
}

// A run that crosses pieces: its first piece's warp adds side 1 of that piece
// and side 0 of the following ones, in order.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const int32_t* __restrict__ keys, int N, int V, int C,
                                                              float scale, void* __restrict__ dtable,
                                                              const float* __restrict__ part) {
  const int lane = threadIdx.x & 31;
  const int parts = (C + kCols - 1) / kCols;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int piece = static_cast<int>(item / parts);
  const int c = static_cast<int>(item % parts) * kCols + lane * 8;
  const int pieces = (N + kPiece - 1) / kPiece;
  if (piece >= pieces - 1) return;
  const int hi = (piece + 1) * kPiece;
  const int key = __ldg(keys + hi - 1);
  if (key >= V || __ldg(keys + hi) != key) return;
  const int lo = piece * kPiece;
  // the run began before this piece: an earlier piece owns it
  if (lo > 0 && __ldg(keys + lo) == key && __ldg(keys + lo - 1) == key) return;
  const int end = lower_bound_warp(keys, N, key + 1);   // one past the run
  const int last = (end - 1) / kPiece;
  if (c >= C) return;
  float acc[8];
  {
    const float4* s = reinterpret_cast<const float4*>(part + (2ll * piece + 1) * C + c);
    const float4 a = s[0], b = s[1];
    acc[0] = a.x; acc[1] = a.y; acc[2] = a.z; acc[3] = a.w;
    acc[4] = b.x; acc[5] = b.y; acc[6] = b.z; acc[7] = b.w;
  }
#pragma unroll 4
  for (int p = piece + 1; p <= last; ++p) {
    const float4* s = reinterpret_cast<const float4*>(part + (2ll * p) * C + c);
    const float4 a = s[0], b = s[1];
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
    acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
  }
  store_row8<kF32>(dtable, static_cast<int64_t>(key) * C + c, acc, scale);
}

// ---- host ------------------------------------------------------------------------
struct SortShape {
  int passes, per, tiles;
};
SortShape sort_shape(int64_t N, int64_t V) {
  SortShape s;
  s.passes = 1;
  while (s.passes < 4 && (V >> (8 * s.passes)) != 0) ++s.passes;   // keys 0..V
  int64_t per = (N + kMaxTiles - 1) / kMaxTiles;
  per = per < kMinTile ? kMinTile : per;
  constexpr int64_t unit = 32 * kSortWarps;
  s.per = static_cast<int>((per + unit - 1) / unit * unit);
  s.tiles = static_cast<int>((N + s.per - 1) / s.per);
  return s;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

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
  const size_t pieces = (n + kPiece - 1) / kPiece;
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
  sort_hist_kernel<<<sh.tiles, kSortThreads, 0, s>>>(tokens, n, v, sh.per, sh.passes, hist);
  st = cuda_status(cudaGetLastError());
  const int32_t *ki = nullptr, *pi = nullptr;
  for (int p = 0; st == TPK_OK && p < sh.passes; ++p) {
    int32_t* ko = buf[(p & 1) * 2];
    int32_t* po = buf[(p & 1) * 2 + 1];
    int32_t* h = hist + static_cast<int64_t>(p) * sh.tiles * kDigits;
    sort_scatter_kernel<<<sh.tiles, kSortThreads, 0, s>>>(tokens, ki, pi, n, v, sh.per, 8 * p, h,
                                                          p + 1 < sh.passes ? h + sh.tiles * kDigits : nullptr, ko, po);
    st = cuda_status(cudaGetLastError());
    ki = ko;
    pi = po;
  }
  if (st != TPK_OK) return st;
  const int64_t pieces = (N + kPiece - 1) / kPiece;
  const int parts = (C + kCols - 1) / kCols;
  const int64_t sum_blocks = (pieces * parts + kThreads / 32 - 1) / (kThreads / 32);
  int64_t zero_blocks = (V + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = int64_t{num_sms()} * 8;
  if (zero_blocks > most) zero_blocks = most;
  if (sum_blocks + zero_blocks > 0x7fffffff) return TPK_E_ARG;
  const unsigned grid = static_cast<unsigned>(sum_blocks + zero_blocks);
  if (f32)
    embed_sum_kernel<true><<<grid, kThreads, 0, s>>>(ki, pi, static_cast<const uint4*>(dout), n, v, C, scale, dtable,
                                                     part, static_cast<int>(sum_blocks));
  else
    embed_sum_kernel<false><<<grid, kThreads, 0, s>>>(ki, pi, static_cast<const uint4*>(dout), n, v, C, scale, dtable,
                                                      part, static_cast<int>(sum_blocks));
  st = cuda_status(cudaGetLastError());
  if (st != TPK_OK || pieces < 2) return st;
  if (f32)
    embed_join_kernel<true><<<static_cast<unsigned>(sum_blocks), kThreads, 0, s>>>(ki, n, v, C, scale, dtable, part);
  else
    embed_join_kernel<false><<<static_cast<unsigned>(sum_blocks), kThreads, 0, s>>>(ki, n, v, C, scale, dtable, part);
  return cuda_status(cudaGetLastError());
}
