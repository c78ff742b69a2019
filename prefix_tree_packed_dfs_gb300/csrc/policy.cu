// Clipped policy objective over a packed batch, with a KL term, and its
// gradient with respect to the vocabulary loss of every forwarded position
// (include/tpk.h has the formulas).
//
// Two passes.  The first walks the raw tokens (or, for ratios of whole
// sequences, a CTA walks each sequence): it forms every token's terms, adds the
// weighted ones up, and leaves the token's share of the gradient.  The second
// adds the shares of the raw tokens of each position, in their order, and joins
// the sums; it starts under the first (programmatic dependent launch).
// Where a weight is zero nothing else of the token is read.
// Log-ratios are differences of two fp32 numbers, formed and compared with the
// clip's borders in fp64, so that a token is never on the wrong side; a
// sequence's mean is an fp64 sum.  exp(t) - t - 1 near t = 0 is its series.
// What bounds it: the launches; the batch of 64 rollouts below moves 4 MB.
#include "pair.cuh"
#include "rowwise.cuh"

namespace tpk {
namespace {

constexpr int kPolThreads = 256;
constexpr int kPolBlocks = 1216;   // of the token pass, at most
constexpr int kStats = 5;          // objective, KL, clipped, ratio, weight

struct Policy {
  const float *loss, *old_logp, *ref_logp, *advantage, *weight;
  const int32_t* token_index;
  const int32_t *raw_begin, *raw;
  const int32_t* offsets;
  int32_t n_seqs;
  int64_t R, F;
  double log_lo, log_hi, log_dual;   // borders of the log-ratio; log_dual = inf: none
  float lo, hi, dual, kl;
  float* share;                      // [R] gradient of each raw token
  double* sums;                      // [blocks][kStats]
  int32_t sum_rows;
  float* stats;
  float* dloss;
};

struct Term {
  float grad;     // of advantage * ratio, times the ratio; 0 where held by a border
  float objective, held;
};
__device__ __forceinline__ Term clipped(const Policy& p, double d, float ratio, float adv) {
  Term t;
  float used = ratio;
  bool held = false;
  if (adv > 0.f) {
    if (d > p.log_hi) held = true, used = p.hi;
  } else if (adv < 0.f) {
    if (d < p.log_lo) held = true, used = p.lo;
    if (d > p.log_dual) held = true, used = p.dual;
  }
  t.objective = -adv * used;
  t.grad = held ? 0.f : adv * ratio;
  t.held = held ? 1.f : 0.f;
  return t;
}

// exp(t) - t - 1
__device__ __forceinline__ float k3(float t) {
  if (fabsf(t) >= 0.3f) return expm1f(t) - t;
  // t^2 (1/2! + t/3! + .. + t^5/7!): the next term is 4e-8 of it
  float s = fmaf(t, 1.f / 5040.f, 1.f / 720.f);
  s = fmaf(t, s, 1.f / 120.f);
  s = fmaf(t, s, 1.f / 24.f);
  s = fmaf(t, s, 1.f / 6.f);
  s = fmaf(t, s, 0.5f);
  return t * t * s;
}

// Position of raw token r, or -1 where r carries no loss.
__device__ __forceinline__ int64_t position(const Policy& p, int64_t r, float& w) {
  w = __ldg(p.weight + r);
  if (w == 0.f) return -1;
  const int64_t f = __ldg(p.token_index + r);
  return f >= 0 && f < p.F ? f : -1;
}

// The block's sums of s into row `row` of p.sums.
template <int kThreadsOf>
__device__ __forceinline__ void put_sums(const Policy& p, const float (&s)[kStats], int row) {
  __shared__ double part[kThreadsOf / 32][kStats];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < kStats; ++i) {
    double v = s[i];
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

// The KL term of a token: its value (weighted sums), its share of the gradient.
__device__ __forceinline__ float kl_of(const Policy& p, int64_t r, float logp, float& grad) {
  const float t = static_cast<float>(static_cast<double>(__ldg(p.ref_logp + r)) - static_cast<double>(logp));
  if (p.kl != 0.f) grad += p.kl * expm1f(t);
  return k3(t);
}

__global__ void __launch_bounds__(kPolThreads) policy_token_kernel(const Policy p) {
  ptx::dependents_launch();
  float s[kStats] = {};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPolThreads;
#pragma unroll 2
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kPolThreads + threadIdx.x; r < p.R; r += step) {
    float w, g = 0.f;
    const int64_t f = position(p, r, w);
    if (f >= 0) {
      const float logp = -__ldg(p.loss + f), adv = __ldg(p.advantage + r);
      const double d = static_cast<double>(logp) - static_cast<double>(__ldg(p.old_logp + r));
      const float ratio = expf(static_cast<float>(d));
      const Term t = clipped(p, d, ratio, adv);
      float objective = t.objective, kl = 0.f;
      g = t.grad;
      if (p.ref_logp) {
        kl = kl_of(p, r, logp, g);
        if (p.kl != 0.f) objective = fmaf(p.kl, kl, objective);
      }
      g *= w;
      s[0] = fmaf(w, objective, s[0]);
      s[1] = fmaf(w, kl, s[1]);
      s[2] = fmaf(w, t.held, s[2]);
      s[3] = fmaf(w, ratio, s[3]);
      s[4] += w;
    }
    p.share[r] = g;
  }
  put_sums<kPolThreads>(p, s, blockIdx.x);
}

template <typename T>
__device__ __forceinline__ T block_sum(T v, T* room) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();   // room has been read
  if (lane == 0) room[warp] = v;
  __syncthreads();
  T s = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) s += room[i];
  return s;
}

// A CTA per sequence: ratio = exp(mean log-ratio of its tokens that carry loss).
constexpr int kSeqThreads = 512;
__global__ void __launch_bounds__(kSeqThreads) policy_sequence_kernel(const Policy p) {
  ptx::dependents_launch();
  __shared__ double room[kSeqThreads / 32];
  auto inside = [&](int64_t x) { return x < 0 ? 0 : x > p.R ? p.R : x; };
  const int i = blockIdx.x;
  const int64_t lo = inside(__ldg(p.offsets + i)), hi = inside(__ldg(p.offsets + i + 1));
  // tokens before the first and after the last sequence carry nothing
  if (i == 0)
    for (int64_t r = threadIdx.x; r < lo; r += kSeqThreads) p.share[r] = 0.f;
  if (i + 1 == p.n_seqs)
    for (int64_t r = hi + threadIdx.x; r < p.R; r += kSeqThreads) p.share[r] = 0.f;
  double sum = 0.0, many = 0.0;
#pragma unroll 4
  for (int64_t r = lo + threadIdx.x; r < hi; r += kSeqThreads) {
    float w;
    const int64_t f = position(p, r, w);
    if (f >= 0) {
      sum -= static_cast<double>(__ldg(p.loss + f)) + static_cast<double>(__ldg(p.old_logp + r));
      many += 1.0;
    }
  }
  sum = block_sum(sum, room);
  many = block_sum(many, room);
  const double d = many > 0.0 ? sum / many : 0.0;
  const float ratio = expf(static_cast<float>(d));
  // the ratio's gradient, which every token shares
  double pull = 0.0;
  float s[kStats] = {};
#pragma unroll 4
  for (int64_t r = lo + threadIdx.x; r < hi; r += kSeqThreads) {
    float w;
    if (position(p, r, w) < 0) continue;
    const Term t = clipped(p, d, ratio, __ldg(p.advantage + r));
    pull += static_cast<double>(w * t.grad);
    s[0] = fmaf(w, t.objective, s[0]);
    s[2] = fmaf(w, t.held, s[2]);
    s[3] = fmaf(w, ratio, s[3]);
    s[4] += w;
  }
  pull = block_sum(pull, room);
  const float each = many > 0.0 ? static_cast<float>(pull / many) : 0.f;
#pragma unroll 4
  for (int64_t r = lo + threadIdx.x; r < hi; r += kSeqThreads) {
    float w, g = 0.f;
    const int64_t f = position(p, r, w);
    if (f >= 0) {
      g = each;
      if (p.ref_logp) {
        float k = 0.f;
        const float kl = kl_of(p, r, -__ldg(p.loss + f), k);
        g = fmaf(w, k, g);
        if (p.kl != 0.f) s[0] = fmaf(w, p.kl * kl, s[0]);
        s[1] = fmaf(w, kl, s[1]);
      }
    }
    p.share[r] = g;
  }
  put_sums<kSeqThreads>(p, s, i);
}

// dloss[f] = sum of the shares of f's raw tokens.  A CTA takes 32 positions,
// one per lane (neighbouring positions' tokens are neighbours in raw order), and
// its eight warps every eighth token of each: a prompt under hundreds of
// sequences is no long walk.  The last CTA joins the first pass's sums.
__global__ void __launch_bounds__(kPolThreads) policy_position_kernel(const Policy p) {
  constexpr int kWarps = kPolThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x + 1 == gridDim.x) {
    ptx::dependency_wait();
    __shared__ double room[kPolThreads / 32];
    for (int i = 0; i < kStats; ++i) {
      double v = 0.0;
      for (int r = threadIdx.x; r < p.sum_rows; r += kPolThreads) v += p.sums[static_cast<int64_t>(r) * kStats + i];
      v = block_sum(v, room);
      if (threadIdx.x == 0) p.stats[i] = static_cast<float>(v);
    }
    return;
  }
  const int64_t f = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  int64_t lo = 0, hi = 0;
  if (f < p.F) {
    lo = __ldg(p.raw_begin + f);
    hi = __ldg(p.raw_begin + f + 1);
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.R ? p.R : hi;
  }
  ptx::dependency_wait();
  float s = 0.f;
#pragma unroll 4
  for (int64_t e = lo + warp; e < hi; e += kWarps) {
    const int64_t r = __ldg(p.raw + e);
    if (r >= 0 && r < p.R) s += __ldcg(p.share + r);
  }
  __shared__ float part[kWarps][32];
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || f >= p.F) return;
#pragma unroll
  for (int i = 1; i < kWarps; ++i) s += part[i][lane];
  p.dloss[f] = s;
}

int token_blocks(int64_t R) {
  const int64_t b = (R + 2 * kPolThreads - 1) / (2 * kPolThreads);
  return static_cast<int>(b < 1 ? 1 : b > kPolBlocks ? kPolBlocks : b);
}
size_t share_bytes(int64_t R) { return (static_cast<size_t>(R) * 4 + 255) / 256 * 256; }

}  // namespace
}  // namespace tpk

extern "C" size_t tpk_policy_loss_workspace_bytes(int64_t R, int32_t n_seqs) {
  using namespace tpk;
  if (R < 0 || R >= (int64_t{1} << 31) || n_seqs < 0) return 0;
  const size_t rows = n_seqs > 0 ? static_cast<size_t>(n_seqs) : token_blocks(R);
  return share_bytes(R) + rows * kStats * sizeof(double);
}

extern "C" int tpk_policy_loss(const float* loss, const float* old_logp, const float* ref_logp, const float* advantage,
                               const float* weight, const int32_t* token_index, const int32_t* fwd_raw_begin,
                               const int32_t* fwd_raw, const int32_t* seq_offsets, int32_t n_seqs,
                               const tpk_policy_opts* opts, float* stats, float* dloss, int64_t R, int64_t F,
                               void* workspace, size_t ws_bytes, void* stream) {
  using namespace tpk;
  if (!opts || R < 0 || F < 0 || F > R || R >= (int64_t{1} << 31) || !stats) return TPK_E_ARG;
  if (seq_offsets ? n_seqs < 1 : n_seqs != 0) return TPK_E_ARG;
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
  p.log_lo = log1p(-opts->clip_low);
  p.log_hi = log1p(opts->clip_high);
  p.log_dual = opts->dual_clip > 0.0 ? log(opts->dual_clip) : INFINITY;
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
  cfg.gridDim = dim3(static_cast<unsigned>((F + 31) / 32 + 1));
  cfg.blockDim = dim3(kPolThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, policy_position_kernel, p));
}
