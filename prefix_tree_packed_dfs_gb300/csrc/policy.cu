// Clipped policy objective over a packed batch, with a KL term, and its
// gradient with respect to the vocabulary loss of every forwarded position
// (include/tpk.h has the formulas).
//
// Two passes.  The first walks the raw tokens (or, for ratios of whole
// sequences, a CTA walks each sequence): it forms every token's terms, adds the
// weighted ones up, and leaves the token's share of the gradient.  The second
// adds the shares of the raw tokens of each position, in their order, and joins
// the sums; it starts under the first (programmatic dependent launch).
// Log-ratios are differences of two fp32 numbers and are kept as the exact sum
// of two, for their comparison with the clip's borders (a token is never on the
// wrong side) and for a sequence's mean, as are the sums of a thread's batches of
// tokens; fp64 instructions, of which this part has few, are left to single threads
// (512 sequences, 548,000 tokens: a sequence pass with fp64 block sums took 83 us,
// this one 13).  exp(t) - t - 1 near t = 0 is its series.
// What bounds it: latency, of the launches and of the chain offset -> token ->
// share (64 sequences, 170,000 tokens: both passes 13.5 us; those 512: 20.2), and in
// long sequences one SM each (8 of 100,000 tokens: 305).
#include <cmath>

#include "pair.cuh"
#include "rowwise.cuh"

namespace tpk {
namespace {

constexpr int kPolThreads = 256;
constexpr int kPolBlocks = 1216;   // of the token pass, at most
constexpr int kStats = 5;          // objective, KL, clipped, ratio, weight

// The unevaluated sum of two fp32 numbers, the second below half a step of the first
// (0 beside an infinity, whose error would come out as NaN).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = a + b, t = s - a, e = (a - (s - t)) + (b - t);
  return Pair{s, e == e ? e : 0.f};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}
// Adds x to s, as exactly as two fp32 numbers can hold it; the second stays below half
// a step of the first, or it would round itself after a million terms alike.
__device__ __forceinline__ void into(Pair& s, float x) {
  const Pair t = two_sum(s.hi, x);
  const float l = s.lo + t.lo, h = t.hi + l, e = l - (h - t.hi);
  s = Pair{h, e == e ? e : 0.f};
}
// a - b, of which the sign is right next to 0 too; NaN, which is on neither side,
// for equal infinities
__device__ __forceinline__ float less(Pair a, Pair b) { return (a.hi - b.hi) + (a.lo - b.lo); }

struct Policy {
  const float *loss, *old_logp, *ref_logp, *advantage, *weight;
  const int32_t* token_index;
  const int32_t *raw_begin, *raw;
  const int32_t* offsets;
  int32_t n_seqs;
  int64_t R, F;
  Pair log_lo, log_hi, log_dual;     // borders of the log-ratio; log_dual = inf: none
  float lo, hi, dual, kl;
  float* share;                      // [R] gradient of each raw token
  double* sums;                      // [rows][kStats]
  int32_t sum_rows;
  float* stats;
  float* dloss;
};

// For a log-ratio: the ratio to use, and whether a border holds it, where the
// advantage is positive (0) and negative (1).
struct Clip {
  float ratio, used[2];
  bool held[2];
};
__device__ __forceinline__ Clip clip_of(const Policy& p, Pair d) {
  Clip c;
  c.ratio = expf(d.hi);
  c.held[0] = less(d, p.log_hi) > 0.f;
  c.used[0] = c.held[0] ? p.hi : c.ratio;
  const bool below = less(d, p.log_lo) < 0.f, above = less(d, p.log_dual) > 0.f;
  c.held[1] = below || above;
  c.used[1] = above ? p.dual : below ? p.lo : c.ratio;
  return c;
}

struct Term {
  float grad;     // of the ratio's part, by the log-ratio; 0 where held by a border
  float objective, held;
};
__device__ __forceinline__ Term term_of(const Clip& c, float adv) {
  // without an advantage nothing, however large the ratio
  const bool neg = adv < 0.f, zero = adv == 0.f;
  const bool held = !zero && (neg ? c.held[1] : c.held[0]);
  Term t;
  t.objective = zero ? 0.f : -adv * (neg ? c.used[1] : c.used[0]);
  t.grad = held || zero ? 0.f : adv * c.ratio;
  t.held = held ? 1.f : 0.f;
  return t;
}

// exp(t) - t - 1; infinite at both infinities
__device__ __forceinline__ float k3(float t) {
  if (fabsf(t) >= 0.3f) {
    const float e = expm1f(t);
    return e == INFINITY ? e : e - t;
  }
  // t^2 (1/2! + t/3! + .. + t^5/7!): the next term is 4e-8 of it
  float s = fmaf(t, 1.f / 5040.f, 1.f / 720.f);
  s = fmaf(t, s, 1.f / 120.f);
  s = fmaf(t, s, 1.f / 24.f);
  s = fmaf(t, s, 1.f / 6.f);
  s = fmaf(t, s, 0.5f);
  return t * t * s;
}

// A raw token: its weight and its position, -1 where it carries no loss.
struct Token {
  float w;
  int32_t f;
};
__device__ __forceinline__ Token token_at(const Policy& p, int64_t r) {
  Token t;
  t.w = __ldg(p.weight + r);
  const int32_t f = __ldg(p.token_index + r);
  t.f = t.w != 0.f && f >= 0 && f < p.F ? f : -1;
  return t;
}

// The KL term of a token; its share of the gradient is added to grad.
__device__ __forceinline__ float kl_of(const Policy& p, float ref, float loss, float& grad) {
  const float t = ref + loss;   // ref - logp
  if (p.kl != 0.f) grad += p.kl * expm1f(t);
  return k3(t);
}

// The block's sums of s into row `row` of p.sums: a thread's is off by the roundings of
// one batch of tokens and one more, however many it had, a warp's by five more.
template <int kThreadsOf>
__device__ __forceinline__ void put_sums(const Policy& p, const Pair (&s)[kStats], int row) {
  __shared__ float part[kThreadsOf / 32][kStats];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < kStats; ++i) {
    float v = s[i].hi + s[i].lo;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) part[warp][i] = v;
  }
  __syncthreads();
  if (threadIdx.x < kStats) {
    double v = 0.0;
    for (int i = 0; i < kThreadsOf / 32; ++i) v += part[i][threadIdx.x];
    p.sums[static_cast<int64_t>(row) * kStats + threadIdx.x] = v;
  }
}

__global__ void __launch_bounds__(kPolThreads) policy_token_kernel(const Policy p) {
  ptx::dependents_launch();
  constexpr int kBatch = 2;
  Pair s[kStats] = {};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPolThreads;
#pragma unroll 1
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kPolThreads + threadIdx.x; r0 < p.R; r0 += kBatch * step) {
    Token k[kBatch];
    float old[kBatch], adv[kBatch], ref[kBatch], loss[kBatch], some[kStats] = {};
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int64_t r = r0 + j * step;
      const bool in = r < p.R;
      k[j] = in ? token_at(p, r) : Token{0.f, -1};
      old[j] = in ? __ldg(p.old_logp + r) : 0.f;
      adv[j] = in ? __ldg(p.advantage + r) : 0.f;
      ref[j] = in && p.ref_logp ? __ldg(p.ref_logp + r) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) loss[j] = k[j].f >= 0 ? __ldg(p.loss + k[j].f) : 0.f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      float g = 0.f;
      if (k[j].f >= 0) {
        const Clip c = clip_of(p, two_sum(-loss[j], -old[j]));
        const Term t = term_of(c, adv[j]);
        float objective = t.objective, kl = 0.f;
        g = t.grad;
        if (p.ref_logp) {
          kl = kl_of(p, ref[j], loss[j], g);
          if (p.kl != 0.f) objective = fmaf(p.kl, kl, objective);
        }
        const float w = k[j].w;
        g *= w;
        some[0] = fmaf(w, objective, some[0]);
        some[1] = fmaf(w, kl, some[1]);
        some[2] = fmaf(w, t.held, some[2]);
        some[3] = fmaf(w, c.ratio, some[3]);
        some[4] += w;
      }
      if (r0 + j * step < p.R) p.share[r0 + j * step] = g;
    }
#pragma unroll
    for (int i = 0; i < kStats; ++i) into(s[i], some[i]);
  }
  put_sums<kPolThreads>(p, s, blockIdx.x);
}

// The warps' sums of v and of n, for the first of them to add up.
template <int kThreadsOf>
struct Parts {
  Pair sum[kThreadsOf / 32];
  int many[kThreadsOf / 32];

  __device__ __forceinline__ void put(Pair v, int n) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v = add(v, Pair{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = v, many[threadIdx.x >> 5] = n;
  }
  __device__ __forceinline__ Pair total(int& n) const {
    Pair v = sum[0];
    n = many[0];
#pragma unroll
    for (int i = 1; i < kThreadsOf / 32; ++i) v = add(v, sum[i]), n += many[i];
    return v;
  }
};

// A CTA per sequence: ratio = exp(mean log-ratio of its tokens that carry loss).
constexpr int kSeqThreads = 256;
__global__ void __launch_bounds__(kSeqThreads, 4) policy_sequence_kernel(const Policy p) {
  ptx::dependents_launch();
  __shared__ Clip clip;
  __shared__ Parts<kSeqThreads> log_ratios, pulls;
  __shared__ float share_of_pull;
  auto inside = [&](int64_t x) { return x < 0 ? 0 : x > p.R ? p.R : x; };
  const int i = blockIdx.x;
  const int64_t lo = inside(__ldg(p.offsets + i)), hi = inside(__ldg(p.offsets + i + 1));
  // tokens before the first and after the last sequence carry nothing
  if (i == 0)
    for (int64_t r = threadIdx.x; r < lo; r += kSeqThreads) p.share[r] = 0.f;
  if (i + 1 == p.n_seqs)
    for (int64_t r = hi + threadIdx.x; r < p.R; r += kSeqThreads) p.share[r] = 0.f;
  // A sequence of up to kKeep tokens per thread is read once; what is longer is
  // read again by each step.
  constexpr int kKeep = 6, kBatch = 4;
  const int64_t first = lo + threadIdx.x, later = first + int64_t{kKeep} * kSeqThreads;
  Token kept[kKeep];
  float old[kKeep], adv[kKeep], ref[kKeep], loss[kKeep];
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int64_t r = first + j * kSeqThreads;
    kept[j] = Token{0.f, -1};
    old[j] = adv[j] = ref[j] = 0.f;
    if (r < hi) {
      kept[j] = token_at(p, r);
      old[j] = __ldg(p.old_logp + r);
      adv[j] = __ldg(p.advantage + r);
      if (p.ref_logp) ref[j] = __ldg(p.ref_logp + r);
    }
  }
#pragma unroll
  for (int j = 0; j < kKeep; ++j) loss[j] = kept[j].f >= 0 ? __ldg(p.loss + kept[j].f) : 0.f;
  Pair sum{0.f, 0.f};
  int many = 0;
#pragma unroll
  for (int j = 0; j < kKeep; ++j)
    if (kept[j].f >= 0) {
      sum = add(sum, two_sum(-loss[j], -old[j]));
      ++many;
    }
#pragma unroll 4
  for (int64_t r = later; r < hi; r += kSeqThreads) {
    const Token k = token_at(p, r);
    const float o = __ldg(p.old_logp + r);
    if (k.f >= 0) {
      sum = add(sum, two_sum(-__ldg(p.loss + k.f), -o));
      ++many;
    }
  }
  log_ratios.put(sum, many);
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = log_ratios.total(many);
    const double d = many ? (static_cast<double>(sum.hi) + static_cast<double>(sum.lo)) / many : 0.0;
    const float top = static_cast<float>(d);
    clip = clip_of(p, Pair{top, isinf(top) ? 0.f : static_cast<float>(d - static_cast<double>(top))});
  }
  __syncthreads();
  const Clip c = clip;
  // the ratio's gradient, which every token shares
  Pair pull{0.f, 0.f};
  // sums of the kept tokens; those of the others are added to them as pairs
  float near[kStats] = {};
  auto gather = [&](const Token& k, float a, float (&to)[kStats]) {
    const Term t = term_of(c, a);
    pull = add(pull, Pair{k.w * t.grad, 0.f});
    to[0] = fmaf(k.w, t.objective, to[0]);
    to[2] = fmaf(k.w, t.held, to[2]);
    to[3] = fmaf(k.w, c.ratio, to[3]);
    to[4] += k.w;
  };
#pragma unroll
  for (int j = 0; j < kKeep; ++j)
    if (kept[j].f >= 0) gather(kept[j], adv[j], near);
  Pair s[kStats];
#pragma unroll
  for (int i = 0; i < kStats; ++i) s[i] = Pair{near[i], 0.f};
#pragma unroll 1
  for (int64_t r0 = later; r0 < hi; r0 += kBatch * kSeqThreads) {
    Token k[kBatch];
    float a[kBatch], some[kStats] = {};
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int64_t r = r0 + j * kSeqThreads;
      k[j] = r < hi ? token_at(p, r) : Token{0.f, -1};
      a[j] = r < hi ? __ldg(p.advantage + r) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (k[j].f >= 0) gather(k[j], a[j], some);
#pragma unroll
    for (int i = 0; i < kStats; ++i) into(s[i], some[i]);
  }
  pulls.put(pull, 0);
  __syncthreads();
  if (threadIdx.x == 0) {
    int unused;
    pull = pulls.total(unused);
    share_of_pull = many ? (pull.hi + pull.lo) / static_cast<float>(many) : 0.f;
  }
  __syncthreads();
  const float each = share_of_pull;
  float kls = 0.f, parts = 0.f;   // sums of w kl, and of its part of the objective
  auto share = [&](const Token& k, float token_ref, float token_loss) {
    if (k.f < 0) return 0.f;
    if (!p.ref_logp) return each;
    float pull_kl = 0.f;
    const float kl = kl_of(p, token_ref, token_loss, pull_kl);
    if (p.kl != 0.f) parts = fmaf(k.w, p.kl * kl, parts);
    kls = fmaf(k.w, kl, kls);
    return fmaf(k.w, pull_kl, each);
  };
#pragma unroll
  for (int j = 0; j < kKeep; ++j)
    if (first + j * kSeqThreads < hi) p.share[first + j * kSeqThreads] = share(kept[j], ref[j], loss[j]);
  into(s[0], parts);
  into(s[1], kls);
#pragma unroll 1
  for (int64_t r0 = later; r0 < hi; r0 += kBatch * kSeqThreads) {
    kls = parts = 0.f;
    Token k[kBatch];
    float of_ref[kBatch], of_loss[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int64_t r = r0 + j * kSeqThreads;
      k[j] = r < hi ? token_at(p, r) : Token{0.f, -1};
      of_ref[j] = p.ref_logp && r < hi ? __ldg(p.ref_logp + r) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) of_loss[j] = p.ref_logp && k[j].f >= 0 ? __ldg(p.loss + k[j].f) : 0.f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (r0 + j * kSeqThreads < hi) p.share[r0 + j * kSeqThreads] = share(k[j], of_ref[j], of_loss[j]);
    into(s[0], parts);
    into(s[1], kls);
  }
  put_sums<kSeqThreads>(p, s, i);
}

// dloss[f] = sum of the shares of f's raw tokens.  A warp takes 32 neighbouring
// positions, one per lane (their tokens are neighbours in raw order too).  Where
// one of the 32 has many tokens (a prompt under hundreds of sequences) the
// CTA's eight warps share each list out.  A CTA's warps take groups from all over
// the batch, so that a prompt's groups meet different CTAs.  The last CTA joins
// the first pass's sums.
constexpr int kLong = 8;   // tokens of a position that a lane adds up alone
constexpr int kQuads = 8;  // 16-byte pieces of a long list in flight

// The shares of up to kMost tokens from e on, short of hi.
template <int kMost>
__device__ __forceinline__ float some_shares(const Policy& p, int e, int hi) {
  int r[kMost];
#pragma unroll
  for (int j = 0; j < kMost; ++j) r[j] = e + j < hi ? __ldg(p.raw + e + j) : -1;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < kMost; ++j)
    if (r[j] >= 0 && r[j] < p.R) s += __ldcg(p.share + r[j]);
  return s;
}
// The lists of neighbouring positions lie far apart: a lane reads its own in
// 16-byte pieces.
__device__ __forceinline__ float many_shares(const Policy& p, int lo, int hi) {
  const int to_line = static_cast<int>(-(reinterpret_cast<intptr_t>(p.raw + lo) >> 2)) & 3;
  const int first = lo + to_line < hi ? lo + to_line : hi;
  float s = some_shares<3>(p, lo, first);
  int e = first;
  for (; e + 4 * kQuads <= hi; e += 4 * kQuads) {
    int4 r[kQuads];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) r[j] = __ldg(reinterpret_cast<const int4*>(p.raw + e) + j);
    float v[4 * kQuads];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int at[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = at[i] >= 0 && at[i] < p.R ? __ldcg(p.share + at[i]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4 * kQuads; ++j) s += v[j];
  }
  for (; e < hi; e += 16) s += some_shares<16>(p, e, hi);
  return s;
}

__global__ void __launch_bounds__(kPolThreads) policy_position_kernel(const Policy p) {
  constexpr int kWarps = kPolThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = static_cast<int>(gridDim.x) - 1;
  if (static_cast<int>(blockIdx.x) == blocks) {
    ptx::dependency_wait();
    __shared__ double room[kStats][32];
    const int i = threadIdx.x / 32;
    if (i < kStats) {
      double v = 0.0;
#pragma unroll 4
      for (int r = lane; r < p.sum_rows; r += 32) v += __ldcg(p.sums + static_cast<int64_t>(r) * kStats + i);
      room[i][lane] = v;
      __syncwarp();
      if (lane == 0) {
        for (int l = 1; l < 32; ++l) v += room[i][l];
        p.stats[i] = static_cast<float>(v);
      }
    }
    return;
  }
  const int64_t f = (static_cast<int64_t>(warp) * blocks + blockIdx.x) * 32 + lane;
  int lo = 0, hi = 0;
  if (f < p.F) {   // (whatever the list's ends are, it stays within [0, R))
    const int most = static_cast<int>(p.R);
    lo = min(max(__ldg(p.raw_begin + f), 0), most);
    hi = min(max(__ldg(p.raw_begin + f + 1), lo), most);
  }
  __shared__ int from[kWarps][32], to[kWarps][32], is_long[kWarps];
  __shared__ float part[kWarps][32];
  from[warp][lane] = lo;
  to[warp][lane] = hi;
  const bool any = __any_sync(0xffffffffu, hi - lo > kLong);
  if (lane == 0) is_long[warp] = any;
  ptx::dependency_wait();
  if (!any && f < p.F) p.dloss[f] = some_shares<kLong>(p, lo, hi);
  __syncthreads();
  for (int g = 0; g < kWarps; ++g) {
    if (!is_long[g]) continue;
    const int first = from[g][lane], n = to[g][lane] - first;
    auto cut = [&](int w) { return first + static_cast<int>(static_cast<int64_t>(n) * w / kWarps); };
    part[warp][lane] = many_shares(p, cut(warp), cut(warp + 1));
    __syncthreads();
    if (warp == g && f < p.F) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += part[i][lane];
      p.dloss[f] = s;
    }
    __syncthreads();
  }
}

int token_blocks(int64_t R) {
  const int64_t b = (R + 2 * kPolThreads - 1) / (2 * kPolThreads);
  return static_cast<int>(b < 1 ? 1 : b > kPolBlocks ? kPolBlocks : b);
}
size_t share_bytes(int64_t R) { return (static_cast<size_t>(R) * 4 + 255) / 256 * 256; }
// Lists and partial sums are walked in strides that run past their ends by less than 8,192, in 32 bits.
bool count_ok(int64_t n) { return n >= 0 && n < (int64_t{1} << 31) - 8192; }

}  // namespace
}  // namespace tpk

extern "C" size_t tpk_policy_loss_workspace_bytes(int64_t R, int32_t n_seqs) {
  using namespace tpk;
  if (!count_ok(R) || !count_ok(n_seqs)) return 0;
  const size_t rows = n_seqs > 0 ? static_cast<size_t>(n_seqs) : token_blocks(R);
  return share_bytes(R) + rows * kStats * sizeof(double);
}

extern "C" int tpk_policy_loss(const float* loss, const float* old_logp, const float* ref_logp, const float* advantage,
                               const float* weight, const int32_t* token_index, const int32_t* fwd_raw_begin,
                               const int32_t* fwd_raw, const int32_t* seq_offsets, int32_t n_seqs,
                               const tpk_policy_opts* opts, float* stats, float* dloss, int64_t R, int64_t F,
                               void* workspace, size_t ws_bytes, void* stream) {
  using namespace tpk;
  if (!opts || !count_ok(R) || F < 0 || F > R || !stats) return TPK_E_ARG;
  if (seq_offsets ? n_seqs < 1 || !count_ok(n_seqs) : n_seqs != 0) return TPK_E_ARG;
  if (!(opts->clip_low >= 0.0 && opts->clip_low <= 1.0) || !(opts->clip_high >= 0.0) ||
      !(opts->dual_clip == 0.0 || opts->dual_clip > 1.0) || !(opts->kl_coef >= 0.0 && opts->kl_coef < INFINITY))
    return TPK_E_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int st;
  if (R == 0) {
    st = check_device();
    return st != TPK_OK ? st : cuda_status(cudaMemsetAsync(stats, 0, kStats * sizeof(float), s));
  }
  if (!loss || !old_logp || !advantage || !weight || !token_index || !fwd_raw_begin || !fwd_raw || !dloss)
    return TPK_E_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      ws_bytes < tpk_policy_loss_workspace_bytes(R, seq_offsets ? n_seqs : 0))
    return TPK_E_WORKSPACE;
  st = check_device();
  if (st != TPK_OK) return st;
  Policy p{};
  p.loss = loss;
  p.old_logp = old_logp;
  p.ref_logp = ref_logp;
  p.advantage = advantage;
  p.weight = weight;
  p.token_index = token_index;
  p.raw_begin = fwd_raw_begin;
  p.raw = fwd_raw;
  p.offsets = seq_offsets;
  p.n_seqs = n_seqs;
  p.R = R;
  p.F = F;
  auto pair = [](double x) {
    const float top = static_cast<float>(x);
    return Pair{top, std::isfinite(top) ? static_cast<float>(x - static_cast<double>(top)) : 0.f};
  };
  p.log_lo = pair(log1p(-opts->clip_low));
  p.log_hi = pair(log1p(opts->clip_high));
  p.log_dual = pair(opts->dual_clip > 0.0 ? log(opts->dual_clip) : INFINITY);
  p.lo = static_cast<float>(1.0 - opts->clip_low);
  p.hi = static_cast<float>(1.0 + opts->clip_high);
  p.dual = static_cast<float>(opts->dual_clip);
  p.kl = static_cast<float>(opts->kl_coef);
  p.share = static_cast<float*>(workspace);
  p.sums = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + share_bytes(R));
  p.sum_rows = seq_offsets ? n_seqs : token_blocks(R);
  p.stats = stats;
  p.dloss = dloss;
  if (seq_offsets)
    policy_sequence_kernel<<<static_cast<unsigned>(n_seqs), kSeqThreads, 0, s>>>(p);
  else
    policy_token_kernel<<<static_cast<unsigned>(p.sum_rows), kPolThreads, 0, s>>>(p);
  st = cuda_status(cudaGetLastError());
  if (st != TPK_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((F + kPolThreads - 1) / kPolThreads + 1));
  cfg.blockDim = dim3(kPolThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, policy_position_kernel, p));
}
