// The norms around a block, fused with the block's gate and the residual add.
//
// Per row of C channels (RMS norms, statistics and sums in fp32):
//   u = y * rstd(y) * w_post            rstd(a) = 1 / sqrt(mean a^2 + eps)
//   r = res + scale * sigmoid(gate) * u
//   x = r * rstd(r) * w_pre             (r before its bf16 rounding)
// Without y, r = res (the norm before the first block); without w_post u = y;
// without gate the sigmoid is 1.  r and x are rounded to bf16 once.
//
// HBM-bound: one pass reads y, res, gate and writes r, x (10 bytes per
// element).  The backward recomputes r from the same inputs instead of
// reading a saved one (the same bytes, and no rounding in between), so it
// reads res, y, gate, dr, dx and writes dres, dy, dgate (16 bytes per
// element).  A row stays in the registers of kT threads, 16 channels each.
// The weights' gradients are column sums: every group of threads keeps its
// own columns' sums over the rows it walks and writes them once, and a second
// kernel adds the groups in order (deterministic).
#include <cuda_bf16.h>

#include "common.cuh"

namespace tpk {
namespace {

constexpr int kVec = 2;   // 16-byte pieces (8 channels) per thread: kT * 16 >= C

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack8(uint4 u, float (&f)[8]) {
  f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xFFFF0000u);
  f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xFFFF0000u);
  f[4] = __uint_as_float(u.z << 16); f[5] = __uint_as_float(u.z & 0xFFFF0000u);
  f[6] = __uint_as_float(u.w << 16); f[7] = __uint_as_float(u.w & 0xFFFF0000u);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + __expf(-g)); }

// Sum of NV values over the kT threads of a group; every thread gets it.  The
// order is fixed.  r: NV * kT/32 shared floats that no other sum uses until
// the group has passed another barrier (so one barrier per sum is enough).
template <int kT, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], float* r, int group, int t) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (kT > 32) {
    constexpr int kW = kT / 32;
    if ((t & 31) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) r[i * kW + (t >> 5)] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kT) : "memory");
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) v[i] += r[i * kW + w];
    }
  }
}

template <int kT>
constexpr int kBlockThreads = kT < 256 ? 256 : kT;

struct NormParams {
  const uint4* res;
  const uint4* y;
  const uint4* gate;
  const float* w_post;
  const float* w_pre;
  uint4* res_out;
  uint4* x;
  int64_t N, ld_y, ld_gate;   // row strides in 16-byte pieces
  int32_t C;
  float scale, eps;
  // backward
  const uint4* dres_out;
  const uint4* dx;
  uint4* dres;
  uint4* dy;
  uint4* dgate;
  int64_t ld_dy, ld_dgate;
  float* part;                // [groups][2][C]: dw_post, dw_pre
};

template <int kT>
__global__ void __launch_bounds__(kBlockThreads<kT>) block_norm_kernel(const NormParams p) {
  constexpr int kGroups = kBlockThreads<kT> / kT;
  __shared__ float red[kGroups][2 * (kT / 32)];
  const int group = threadIdx.x / kT, t = threadIdx.x % kT;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  if (row >= p.N) return;   // whole groups leave; barriers are per group
  const int vecs = p.C / 8;
  const float inv_c = 1.f / static_cast<float>(p.C);
  uint4 rr[kVec], yy[kVec], gg[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int c = t + j * kT;
    rr[j] = yy[j] = gg[j] = make_uint4(0, 0, 0, 0);
    if (c < vecs) {
      rr[j] = p.res[row * vecs + c];
      if (p.y) yy[j] = p.y[row * p.ld_y + c];
      if (p.gate) gg[j] = p.gate[row * p.ld_gate + c];
    }
  }
  float rstd_y = 1.f;
  if (p.w_post) {
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float a[8];
      unpack8(yy[j], a);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[0] = fmaf(a[e], a[e], ss[0]);
    }
    group_sum<kT, 1>(ss, red[group], group, t);
    rstd_y = rsqrtf(ss[0] * inv_c + p.eps);
  }
  float r[kVec][8];
  float ss[1] = {0.f};
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int c = t + j * kT;
    unpack8(rr[j], r[j]);
    if (c < vecs && p.y) {
      float a[8], w[8];
      unpack8(yy[j], a);
      if (p.w_post) {
        load8(p.w_post + c * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = a[e] * rstd_y * w[e];
      }
      if (p.gate) {
        unpack8(gg[j], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] *= sigmoid(w[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] = fmaf(p.scale, a[e], r[j][e]);
      p.res_out[row * vecs + c] = pack8(r[j]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[0] = fmaf(r[j][e], r[j][e], ss[0]);
  }
  group_sum<kT, 1>(ss, red[group] + kT / 32, group, t);
  const float rstd = rsqrtf(ss[0] * inv_c + p.eps);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int c = t + j * kT;
    if (c >= vecs) continue;
    float w[8];
    load8(p.w_pre + c * 8, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= r[j][e] * rstd;
    p.x[row * vecs + c] = pack8(w);
  }
}

// With rh = r * rstd(r) and dn = dx * w_pre:
//   dr = rstd(r) * (dn - rh * mean(dn * rh)) + dres_out,   dw_pre = sum dx * rh
//   dres = dr;  d = scale * dr;  dgate = d * u * s * (1 - s), s = sigmoid(gate)
//   du = d * s;  with yh = y * rstd(y), dm = du * w_post:
//   dy = rstd(y) * (dm - yh * mean(dm * yh)),              dw_post = sum du * yh
template <int kT>
__global__ void __launch_bounds__(kBlockThreads<kT>) block_norm_bwd_kernel(const NormParams p) {
  constexpr int kGroups = kBlockThreads<kT> / kT;
  constexpr int kW = kT / 32;
  __shared__ float red[kGroups][6 * kW];   // sums of y^2, of dm * yh, and of a row's pair, by turns of rows
  const int group = threadIdx.x / kT, t = threadIdx.x % kT;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * kGroups;
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const int vecs = p.C / 8;
  const float inv_c = 1.f / static_cast<float>(p.C);
  float acc_post[kVec][8] = {}, acc_pre[kVec][8] = {};
  int turn = 0;
  for (int64_t row = gid; row < p.N; row += groups, turn ^= 1) {
    uint4 rr[kVec], yy[kVec], gg[kVec], dd[kVec], xx[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = t + j * kT;
      rr[j] = yy[j] = gg[j] = dd[j] = xx[j] = make_uint4(0, 0, 0, 0);
      if (c < vecs) {
        if (p.y) yy[j] = p.y[row * p.ld_y + c];
        rr[j] = p.res[row * vecs + c];
        if (p.gate) gg[j] = p.gate[row * p.ld_gate + c];
        xx[j] = p.dx[row * vecs + c];
        if (p.dres_out) dd[j] = p.dres_out[row * vecs + c];
      }
    }
    float rstd_y = 1.f;
    if (p.w_post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        float a[8];
        unpack8(yy[j], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] = fmaf(a[e], a[e], ss[0]);
      }
      group_sum<kT, 1>(ss, red[group], group, t);
      rstd_y = rsqrtf(ss[0] * inv_c + p.eps);
    }
    float r[kVec][8];
    float s2[2] = {0.f, 0.f};   // sum r^2, sum dn * r
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = t + j * kT;
      unpack8(rr[j], r[j]);
      if (c >= vecs) continue;
      float a[8], w[8];
      if (p.y) {
        unpack8(yy[j], a);
        if (p.w_post) {
          load8(p.w_post + c * 8, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) a[e] = a[e] * rstd_y * w[e];
        }
        if (p.gate) {
          unpack8(gg[j], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) a[e] *= sigmoid(w[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] = fmaf(p.scale, a[e], r[j][e]);
      }
      load8(p.w_pre + c * 8, w);
      unpack8(xx[j], a);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s2[0] = fmaf(r[j][e], r[j][e], s2[0]);
        s2[1] = fmaf(a[e] * w[e], r[j][e], s2[1]);
      }
    }
    group_sum<kT, 2>(s2, red[group] + (2 + 2 * turn) * kW, group, t);
    const float rstd = rsqrtf(s2[0] * inv_c + p.eps);
    const float mean_r = s2[1] * inv_c * rstd;   // mean(dn * rh)
    float dm[kVec][8];                           // dm = du * w_post (du without w_post)
    float s1[1] = {0.f};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = t + j * kT;
      if (c >= vecs) continue;
      float w[8], x[8], d[8];
      load8(p.w_pre + c * 8, w);
      unpack8(xx[j], x);
      unpack8(dd[j], d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float rh = r[j][e] * rstd;
        acc_pre[j][e] = fmaf(x[e], rh, acc_pre[j][e]);
        d[e] += rstd * (x[e] * w[e] - rh * mean_r);
      }
      p.dres[row * vecs + c] = pack8(d);
      if (!p.y) continue;
      float a[8], u[8];
      unpack8(yy[j], a);
      if (p.w_post) load8(p.w_post + c * 8, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] *= p.scale;
        a[e] *= rstd_y;                          // yh (y itself without w_post)
        u[e] = p.w_post ? a[e] * w[e] : a[e];
      }
      if (p.gate) {
        float g[8];
        unpack8(gg[j], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = sigmoid(g[e]);
          g[e] = d[e] * u[e] * s * (1.f - s);
          d[e] *= s;
        }
        p.dgate[row * p.ld_dgate + c] = pack8(g);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc_post[j][e] = fmaf(d[e], a[e], acc_post[j][e]);
        dm[j][e] = p.w_post ? d[e] * w[e] : d[e];
        s1[0] = fmaf(dm[j][e], a[e], s1[0]);
      }
    }
    if (!p.y) continue;
    float mean_y = 0.f;
    if (p.w_post) {
      group_sum<kT, 1>(s1, red[group] + kW, group, t);
      mean_y = s1[0] * inv_c;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = t + j * kT;
      if (c >= vecs) continue;
      if (p.w_post) {
        float a[8];
        unpack8(yy[j], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) dm[j][e] = rstd_y * (dm[j][e] - a[e] * rstd_y * mean_y);
      }
      p.dy[row * p.ld_dy + c] = pack8(dm[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int c = t + j * kT;
    if (c >= vecs) continue;
    float4* d = reinterpret_cast<float4*>(p.part + (gid * 2) * p.C + c * 8);
    d[0] = make_float4(acc_post[j][0], acc_post[j][1], acc_post[j][2], acc_post[j][3]);
    d[1] = make_float4(acc_post[j][4], acc_post[j][5], acc_post[j][6], acc_post[j][7]);
    d = reinterpret_cast<float4*>(p.part + (gid * 2 + 1) * p.C + c * 8);
    d[0] = make_float4(acc_pre[j][0], acc_pre[j][1], acc_pre[j][2], acc_pre[j][3]);
    d[1] = make_float4(acc_pre[j][4], acc_pre[j][5], acc_pre[j][6], acc_pre[j][7]);
  }
}

// dw[c] = sum over the groups' partials, 8 warps over the groups and 32
// columns per block, combined in a fixed order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* __restrict__ part, int64_t groups, int C,
                                                      float* __restrict__ dw_post, float* __restrict__ dw_pre) {
  __shared__ float sm[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dw_pre : dw_post;
  if (!out) return;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int64_t g = w; g < groups; g += 8) s += __ldg(part + (g * 2 + blockIdx.y) * C + c);
  }
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sm[i][lane];
    out[c] = s;
  }
}

constexpr int kMaxC = 16384;

int threads_for(int C) {
  const int vecs = C / 8;
  int t = 32;
  while (t * kVec < vecs) t *= 2;
  return t;
}

// Groups of the backward: enough CTAs to fill the SMs, no more than rows.
template <int kT>
int64_t bwd_blocks(int64_t N, int sms) {
  constexpr int kGroups = kBlockThreads<kT> / kT;
  const int64_t want = (N + kGroups - 1) / kGroups;
  const int64_t most = int64_t{sms} * (kT >= 1024 ? 1 : 2);
  return want < most ? want : most;
}
int64_t bwd_groups(int64_t N, int C, int sms) {
  switch (threads_for(C)) {
    case 32: return bwd_blocks<32>(N, sms) * 8;
    case 64: return bwd_blocks<64>(N, sms) * 4;
    case 128: return bwd_blocks<128>(N, sms) * 2;
    case 256: return bwd_blocks<256>(N, sms);
    case 512: return bwd_blocks<512>(N, sms);
    default: return bwd_blocks<1024>(N, sms);
  }
}

template <int kT>
int launch_fwd(const NormParams& p, cudaStream_t s) {
  constexpr int kGroups = kBlockThreads<kT> / kT;
  const int64_t blocks = (p.N + kGroups - 1) / kGroups;
  block_norm_kernel<kT><<<static_cast<unsigned>(blocks), kBlockThreads<kT>, 0, s>>>(p);
  return cuda_status(cudaGetLastError());
}
template <int kT>
int launch_bwd(const NormParams& p, int sms, cudaStream_t s) {
  block_norm_bwd_kernel<kT><<<static_cast<unsigned>(bwd_blocks<kT>(p.N, sms)), kBlockThreads<kT>, 0, s>>>(p);
  return cuda_status(cudaGetLastError());
}

bool rows_ok(const void* p, int64_t ld, int32_t C) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (!p || (ld >= C && ld % 8 == 0));
}

// The rules both directions share; 0 or an error.
int check(const void* res, const void* y, int64_t ld_y, const void* gate, int64_t ld_gate, const float* w_post,
          const float* w_pre, int64_t N, int32_t C, float scale, float eps) {
  if (N < 0 || N >= (int64_t{1} << 31) || C < 8 || C % 8 || !(eps >= 0.f) || !(scale == scale)) return TPK_E_ARG;
  if (C > kMaxC) return TPK_E_UNSUPPORTED;
  if (N > 0 && !y && (gate || w_post)) return TPK_E_ARG;   // tensors of no rows may have no address
  if (!w_pre || reinterpret_cast<uintptr_t>(w_pre) % 16 || reinterpret_cast<uintptr_t>(w_post) % 16) return TPK_E_ARG;
  if (N > 0 && !res) return TPK_E_ARG;
  if (!rows_ok(res, C, C) || !rows_ok(y, ld_y, C) || !rows_ok(gate, ld_gate, C)) return TPK_E_ARG;
  return TPK_OK;
}

}  // namespace
}  // namespace tpk

extern "C" int tpk_block_norm(const void* res, const void* y, int64_t ld_y, const void* gate, int64_t ld_gate,
                              const float* w_post, const float* w_pre, void* res_out, void* x, int64_t N, int32_t C,
                              float scale, float eps, void* stream) {
  using namespace tpk;
  int st = check(res, y, ld_y, gate, ld_gate, w_post, w_pre, N, C, scale, eps);
  if (st != TPK_OK) return st;
  if (N == 0) return TPK_OK;
  if (!x || (y && !res_out) || !rows_ok(x, C, C) || !rows_ok(res_out, C, C)) return TPK_E_ARG;
  st = check_device();
  if (st != TPK_OK) return st;
  NormParams p{};
  p.res = static_cast<const uint4*>(res);
  p.y = static_cast<const uint4*>(y);
  p.gate = static_cast<const uint4*>(gate);
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.res_out = static_cast<uint4*>(res_out);
  p.x = static_cast<uint4*>(x);
  p.N = N;
  p.ld_y = ld_y / 8;
  p.ld_gate = ld_gate / 8;
  p.C = C;
  p.scale = scale;
  p.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (threads_for(C)) {
    case 32: return launch_fwd<32>(p, s);
    case 64: return launch_fwd<64>(p, s);
    case 128: return launch_fwd<128>(p, s);
    case 256: return launch_fwd<256>(p, s);
    case 512: return launch_fwd<512>(p, s);
    default: return launch_fwd<1024>(p, s);
  }
}

// The partials of dw: the widest grid any device of this kind gets (the
// groups actually launched are counted on the device at hand, never more).
extern "C" size_t tpk_block_norm_bwd_workspace_bytes(int64_t N, int32_t C) {
  using namespace tpk;
  if (N < 0 || C < 8 || C % 8 || C > kMaxC) return 0;
  return static_cast<size_t>(bwd_groups(N, C, kMaxSms)) * 2 * static_cast<size_t>(C) * 4;
}

extern "C" int tpk_block_norm_bwd(const void* res, const void* y, int64_t ld_y, const void* gate, int64_t ld_gate,
                                  const float* w_post, const float* w_pre, const void* dres_out, const void* dx,
                                  void* dres, void* dy, int64_t ld_dy, void* dgate, int64_t ld_dgate, float* dw_post,
                                  float* dw_pre, int64_t N, int32_t C, float scale, float eps, void* workspace,
                                  size_t ws_bytes, void* stream) {
  using namespace tpk;
  int st = check(res, y, ld_y, gate, ld_gate, w_post, w_pre, N, C, scale, eps);
  if (st != TPK_OK) return st;
  if (!dw_pre || (w_post != nullptr) != (dw_post != nullptr)) return TPK_E_ARG;
  if (N > 0) {
    if (!dx || !dres || (y != nullptr) != (dy != nullptr) || (gate != nullptr) != (dgate != nullptr)) return TPK_E_ARG;
    if (!rows_ok(dx, C, C) || !rows_ok(dres, C, C) || !rows_ok(dres_out, C, C) || !rows_ok(dy, ld_dy, C) ||
        !rows_ok(dgate, ld_dgate, C))
      return TPK_E_ARG;
    if (!workspace || ws_bytes < tpk_block_norm_bwd_workspace_bytes(N, C) ||
        reinterpret_cast<uintptr_t>(workspace) % 256)
      return TPK_E_WORKSPACE;
  }
  st = check_device();
  if (st != TPK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = num_sms() < kMaxSms ? num_sms() : kMaxSms;
  if (N > 0) {
    NormParams p{};
    p.res = static_cast<const uint4*>(res);
    p.y = static_cast<const uint4*>(y);
    p.gate = static_cast<const uint4*>(gate);
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.N = N;
    p.ld_y = ld_y / 8;
    p.ld_gate = ld_gate / 8;
    p.C = C;
    p.scale = scale;
    p.eps = eps;
    p.dres_out = static_cast<const uint4*>(dres_out);
    p.dx = static_cast<const uint4*>(dx);
    p.dres = static_cast<uint4*>(dres);
    p.dy = static_cast<uint4*>(dy);
    p.dgate = static_cast<uint4*>(dgate);
    p.ld_dy = ld_dy / 8;
    p.ld_dgate = ld_dgate / 8;
    p.part = static_cast<float*>(workspace);
    switch (threads_for(C)) {
      case 32: st = launch_bwd<32>(p, sms, s); break;
      case 64: st = launch_bwd<64>(p, sms, s); break;
      case 128: st = launch_bwd<128>(p, sms, s); break;
      case 256: st = launch_bwd<256>(p, sms, s); break;
      case 512: st = launch_bwd<512>(p, sms, s); break;
      default: st = launch_bwd<1024>(p, sms, s); break;
    }
    if (st != TPK_OK) return st;
  }
  const int64_t groups = N > 0 ? bwd_groups(N, C, sms) : 0;
  norm_dw_kernel<<<dim3((C + 31) / 32, 2), 256, 0, s>>>(static_cast<const float*>(workspace), groups, C, dw_post,
                                                       dw_pre);
  return cuda_status(cudaGetLastError());
}
