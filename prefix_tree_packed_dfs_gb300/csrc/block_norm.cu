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
// element).  In the forward a row stays in the registers of kT threads, 16
// channels each; in the backward it is copied ahead into shared memory.
// The weights' gradients are column sums: every CTA keeps its threads'
// columns' sums over the rows it walks and writes them once, and a second
// kernel adds the CTAs' in order (deterministic).
// Measured on GB300: forward 96,888 x 2,048 283 us, 7.0 TB/s (the copy peak);
// backward 32,768 x 4,096 351 us, 6.1 TB/s (0.90 of it), 77% of the DRAM
// cycles.  What took the backward there from 614 us: rows copied ahead 417,
// then the weights in shared memory instead of L1 340 (packed arithmetic
// alone changed nothing, but its registers are fewer).  One 16-byte piece per
// thread and 512 threads per row instead of two and 256: 449.  Keeping e^-gate
// for an exact 1 - sigmoid costs 3%; the gate read a second time for it 5%, the
// smaller of sigmoid and its complement kept with a sign 7%.
#include <type_traits>

#include "ptx.cuh"
#include "rowwise.cuh"

namespace tpk {
namespace {

constexpr int kVec = 2;   // 16-byte pieces (8 channels) per thread: kT * 16 >= C

__device__ __forceinline__ void unpack8(uint4 u, float (&f)[8]) {
  f[0] = lo16(u.x); f[1] = hi16(u.x);
  f[2] = lo16(u.y); f[3] = hi16(u.y);
  f[4] = lo16(u.z); f[5] = hi16(u.z);
  f[6] = lo16(u.w); f[7] = hi16(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
// 1 / (1 + e^-g) from the hardware's 2^x and reciprocal (each within about
// one ulp; e^-g = inf gives 0): relative error a few 2^-23 plus |g| 2^-24.
__device__ __forceinline__ float sigmoid(float g) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ptx::ex2(g * -1.4426950408889634f)));
  return r;
}
// 8 channels as four packed fp32 pairs: the backward does some 50 operations
// per channel, and a pair takes one instruction and fewer registers.
struct Oct {
  uint64_t v[4];
};
__device__ __forceinline__ uint64_t pair_of(uint32_t u) {
  return ptx::f2(lo16(u), hi16(u));
}
__device__ __forceinline__ Oct oct(uint4 u) { return {{pair_of(u.x), pair_of(u.y), pair_of(u.z), pair_of(u.w)}}; }
__device__ __forceinline__ Oct load_oct(const float* p) {
  const ulonglong2* q = reinterpret_cast<const ulonglong2*>(p);
  const ulonglong2 a = __ldg(q), b = __ldg(q + 1);
  return {{a.x, a.y, b.x, b.y}};
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
  float a, b;
  ptx::unf2(v, a, b);
  return pack2(a, b);
}
__device__ __forceinline__ uint4 pack_oct(const Oct& o) {
  return make_uint4(pack_pair(o.v[0]), pack_pair(o.v[1]), pack_pair(o.v[2]), pack_pair(o.v[3]));
}
__device__ __forceinline__ uint64_t both(float a) { return ptx::f2(a, a); }
__device__ __forceinline__ float add_pair(uint64_t v) {
  float a, b;
  ptx::unf2(v, a, b);
  return a + b;
}
// e^-g of a gate, finite; sigmoid(g) = 1 / (1 + e^-g) of it, and 1 - sigmoid(g)
// as their product: from sigmoid(g) itself it would cancel where that is near 1.
// (Where e^-g would be infinite the sigmoid comes out as zero, and the product too.)
__device__ __forceinline__ uint64_t exp_minus2(uint64_t g) {
  auto finite = [](float e) {   // NaN stays NaN
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(e), "f"(3.4e38f));
    return r;
  };
  float a, b;
  ptx::unf2(ptx::mul2(g, both(-1.4426950408889634f)), a, b);
  return ptx::f2(finite(ptx::ex2(a)), finite(ptx::ex2(b)));
}
__device__ __forceinline__ uint64_t sigmoid2(uint64_t exp_minus) {
  float a, b;
  ptx::unf2(ptx::add2(exp_minus, both(1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return ptx::f2(a, b);
}

// 16 bytes from global to this thread's own place in shared memory.
__device__ __forceinline__ void copy16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

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
  float* part;                // [CTAs][2][C]: dw_post, dw_pre
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
// A group walks rows a fixed stride apart.  A thread reads the same columns
// of every row, so it copies its part of the row after next into its own
// places in shared memory (asynchronously, no barrier) while the group works
// on the current one: the three sums of a row each need a barrier, and
// without the copies ahead nothing is in flight meanwhile.
constexpr int kInputs = 5;   // y, res, gate, dx, dres_out

template <int kT, int kV>
struct BwdShape {
  static constexpr int kGroups = kT < 256 ? 256 / kT : 1;
  static constexpr int kBlock = kGroups * kT;
  static constexpr int kMinBlocks = kBlock * kV <= 256 ? 3 : kBlock * kV <= 512 ? 2 : 1;
  static constexpr int kAhead = kV <= 2 ? 2 : 1;   // rows copied ahead (as shared memory allows)
  // the weights of a thread's columns stay in shared memory too: next to the
  // rows they leave the L1 cache too small to hold them (re-read from L2 for
  // every row otherwise); the widest rows have no room
  static constexpr bool kHoldWeights = kV <= 2;
  static constexpr size_t kRing = static_cast<size_t>(kAhead) * kInputs * kV * kBlock * 16;
  static constexpr size_t kSmem = kRing + (kHoldWeights ? static_cast<size_t>(4) * kV * kBlock * 16 : 0);
};

template <int kT, int kV>
__global__ void __launch_bounds__(BwdShape<kT, kV>::kBlock, BwdShape<kT, kV>::kMinBlocks)
    block_norm_bwd_kernel(const NormParams p) {
  using Shape = BwdShape<kT, kV>;
  constexpr int kW = kT / 32, kBlock = Shape::kBlock, kGroups = Shape::kGroups, kAhead = Shape::kAhead;
  extern __shared__ uint4 ring[];          // [kAhead][kInputs][kV][kBlock]
  __shared__ float red[kGroups][6 * kW];   // sums of y^2, of dm * yh, and of a row's pair, by turns of rows
  const int group = threadIdx.x / kT, t = threadIdx.x % kT;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * kGroups;
  const int vecs = p.C / 8;
  const float inv_c = 1.f / static_cast<float>(p.C);
  uint4* mine = ring + threadIdx.x;
  auto place = [&](int stage, int input, int j) { return mine + ((stage * kInputs + input) * kV + j) * kBlock; };
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.N) {
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const int c = t + j * kT;
        if (c >= vecs) continue;
        if (p.y) copy16(place(stage, 0, j), p.y + row * p.ld_y + c);
        copy16(place(stage, 1, j), p.res + row * vecs + c);
        if (p.gate) copy16(place(stage, 2, j), p.gate + row * p.ld_gate + c);
        copy16(place(stage, 3, j), p.dx + row * vecs + c);
        if (p.dres_out) copy16(place(stage, 4, j), p.dres_out + row * vecs + c);
      }
    }
    copy_commit();
  };
  // [post 0, post 1, pre 0, pre 1][kV][kBlock] pieces of four weights
  uint4* held = ring + Shape::kRing / 16 + threadIdx.x;
  if constexpr (Shape::kHoldWeights) {
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int c = t + j * kT;
      if (c >= vecs) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* w = i < 2 ? p.w_post : p.w_pre;
        if (w) held[(i * kV + j) * kBlock] = __ldg(reinterpret_cast<const uint4*>(w + c * 8) + (i & 1));
      }
    }
  }
  auto weights = [&](bool pre, int j) -> Oct {
    if constexpr (Shape::kHoldWeights) {
      const ulonglong2 a = ptx::lds128u(held + ((2 * pre) * kV + j) * kBlock);
      const ulonglong2 b = ptx::lds128u(held + ((2 * pre + 1) * kV + j) * kBlock);
      return {{a.x, a.y, b.x, b.y}};
    } else {
      return load_oct((pre ? p.w_pre : p.w_post) + (t + j * kT) * 8);
    }
  };
  Oct acc_post[kV] = {}, acc_pre[kV] = {};
  int stage = 0, turn = 0;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  for (int i = 0; i < kAhead; ++i) fetch(first + i * groups, i);
  for (int64_t row = first; row < p.N; row += groups, stage = (stage + 1) % kAhead, turn ^= 1) {
    copy_wait<kAhead - 1>();
    float rstd_y = 1.f;
    if (p.w_post) {
      uint64_t q = 0;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        if (t + j * kT >= vecs) continue;
        const Oct y = oct(*place(stage, 0, j));
#pragma unroll
        for (int e = 0; e < 4; ++e) q = ptx::fma2(y.v[e], y.v[e], q);
      }
      float ss[1] = {add_pair(q)};
      group_sum<kT, 1>(ss, red[group], group, t);
      rstd_y = rsqrtf(ss[0] * inv_c + p.eps);
    }
    Oct r[kV], ex[kV];
    uint64_t q0 = 0, q1 = 0;   // sum r^2, sum dn * r
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int c = t + j * kT;
      if (c >= vecs) continue;
      r[j] = oct(*place(stage, 1, j));
      if (p.y) {
        Oct u = oct(*place(stage, 0, j));
        if (p.w_post) {
          const Oct w = weights(false, j);
#pragma unroll
          for (int e = 0; e < 4; ++e) u.v[e] = ptx::mul2(ptx::mul2(u.v[e], both(rstd_y)), w.v[e]);
        }
        if (p.gate) {
          const Oct g = oct(*place(stage, 2, j));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ex[j].v[e] = exp_minus2(g.v[e]);
            u.v[e] = ptx::mul2(u.v[e], sigmoid2(ex[j].v[e]));
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) r[j].v[e] = ptx::fma2(both(p.scale), u.v[e], r[j].v[e]);
      }
      const Oct w = weights(true, j), x = oct(*place(stage, 3, j));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q0 = ptx::fma2(r[j].v[e], r[j].v[e], q0);
        q1 = ptx::fma2(ptx::mul2(x.v[e], w.v[e]), r[j].v[e], q1);
      }
    }
    float s2[2] = {add_pair(q0), add_pair(q1)};
    group_sum<kT, 2>(s2, red[group] + (2 + 2 * turn) * kW, group, t);
    const float rstd = rsqrtf(s2[0] * inv_c + p.eps);
    const float mean_r = s2[1] * inv_c * rstd;   // mean(dn * rh)
    uint64_t q2 = 0;                             // sum dm * yh
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int c = t + j * kT;
      if (c >= vecs) continue;
      Oct d = {};
      if (p.dres_out) d = oct(*place(stage, 4, j));
      {
        const Oct w = weights(true, j), x = oct(*place(stage, 3, j));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t rh = ptx::mul2(r[j].v[e], both(rstd));
          acc_pre[j].v[e] = ptx::fma2(x.v[e], rh, acc_pre[j].v[e]);
          const uint64_t m = ptx::fma2(rh, both(-mean_r), ptx::mul2(x.v[e], w.v[e]));
          d.v[e] = ptx::fma2(m, both(rstd), d.v[e]);
        }
      }
      p.dres[row * vecs + c] = pack_oct(d);
      if (!p.y) continue;
      Oct yh = oct(*place(stage, 0, j));
      Oct w = {};
      if (p.w_post) w = weights(false, j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        d.v[e] = ptx::mul2(d.v[e], both(p.scale));
        yh.v[e] = ptx::mul2(yh.v[e], both(rstd_y));   // y itself without w_post
      }
      if (p.gate) {
        Oct g;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t s = sigmoid2(ex[j].v[e]), u = p.w_post ? ptx::mul2(yh.v[e], w.v[e]) : yh.v[e];
          d.v[e] = ptx::mul2(d.v[e], s);
          g.v[e] = ptx::mul2(ptx::mul2(d.v[e], u), ptx::mul2(ex[j].v[e], s));
        }
        p.dgate[row * p.ld_dgate + c] = pack_oct(g);
      }
      // from here r holds dm = du * w_post (du without w_post)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc_post[j].v[e] = ptx::fma2(d.v[e], yh.v[e], acc_post[j].v[e]);
        r[j].v[e] = p.w_post ? ptx::mul2(d.v[e], w.v[e]) : d.v[e];
        q2 = ptx::fma2(r[j].v[e], yh.v[e], q2);
      }
    }
    if (p.y) {
      float mean_y = 0.f;
      if (p.w_post) {
        float s1[1] = {add_pair(q2)};
        group_sum<kT, 1>(s1, red[group] + kW, group, t);
        mean_y = s1[0] * inv_c;
      }
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const int c = t + j * kT;
        if (c >= vecs) continue;
        if (p.w_post) {
          const Oct y = oct(*place(stage, 0, j));
          const float k = -rstd_y * mean_y;
#pragma unroll
          for (int e = 0; e < 4; ++e) r[j].v[e] = ptx::mul2(ptx::fma2(y.v[e], both(k), r[j].v[e]), both(rstd_y));
        }
        p.dy[row * p.ld_dy + c] = pack_oct(r[j]);
      }
    }
    fetch(row + kAhead * groups, stage);   // this thread has read its places of the stage
  }
  copy_wait<0>();
  // one partial row per CTA: its groups' sums added in order
  const int64_t width = 2 * static_cast<int64_t>(p.C);
  float* part = p.part + blockIdx.x * width;
  if constexpr (kGroups > 1) {
    float* sums = reinterpret_cast<float*>(ring);   // [kGroups][2][kT * kV * 8]
    constexpr int kRow = kT * kV * 8;
    static_assert(static_cast<size_t>(kGroups) * 2 * kRow * 4 <= Shape::kRing, "sums fit the ring");
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = (t + j * kT) * 8 + 2 * e;
        *reinterpret_cast<uint64_t*>(sums + (group * 2) * kRow + at) = acc_post[j].v[e];
        *reinterpret_cast<uint64_t*>(sums + (group * 2 + 1) * kRow + at) = acc_pre[j].v[e];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.C; i += kBlock) {
      const int which = i >= p.C, c = i - which * p.C;
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) s += sums[(g * 2 + which) * kRow + c];
      part[i] = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int c = t + j * kT;
      if (c >= vecs) continue;
      ulonglong2* d = reinterpret_cast<ulonglong2*>(part + c * 8);
      d[0] = make_ulonglong2(acc_post[j].v[0], acc_post[j].v[1]);
      d[1] = make_ulonglong2(acc_post[j].v[2], acc_post[j].v[3]);
      d = reinterpret_cast<ulonglong2*>(part + p.C + c * 8);
      d[0] = make_ulonglong2(acc_pre[j].v[0], acc_pre[j].v[1]);
      d[1] = make_ulonglong2(acc_pre[j].v[2], acc_pre[j].v[3]);
    }
  }
}

// dw[c] = sum over the CTAs' partials: 32 columns per block, 32 warps over the
// partials, combined in a fixed order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int parts, int C,
                                                       float* __restrict__ dw_post, float* __restrict__ dw_pre) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dw_pre : dw_post;
  if (!out) return;
  float s = 0.f;
  if (c < C) {
#pragma unroll 4
    for (int g = w; g < parts; g += 32) s += __ldg(part + (static_cast<int64_t>(g) * 2 + blockIdx.y) * C + c);
  }
  sm[w][lane] = s;
  __syncthreads();
  s = sm[lane][w];   // column w of the block, partial sum `lane`
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + w < C) out[blockIdx.x * 32 + w] = s;
}

constexpr int kMaxC = 16384;

int threads_for(int C) {
  const int vecs = C / 8;
  int t = 32;
  while (t * kVec < vecs) t *= 2;
  return t;
}

// The backward's shapes by width: threads per row and 16-byte pieces per thread.
template <typename F>
auto bwd_shape(int C, F f) {
  const int vecs = C / 8;
  if (vecs <= 32) return f(BwdShape<32, 1>{}, std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  if (vecs <= 64) return f(BwdShape<64, 1>{}, std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (vecs <= 128) return f(BwdShape<128, 1>{}, std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
  if (vecs <= 256) return f(BwdShape<256, 1>{}, std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (vecs <= 512) return f(BwdShape<256, 2>{}, std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (vecs <= 1024) return f(BwdShape<512, 2>{}, std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  return f(BwdShape<512, 4>{}, std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{});
}

// CTAs of the backward: as many as run together, no more than the rows need.
template <typename Shape>
int64_t bwd_blocks(int64_t N, int sms) {
  const int64_t want = (N + Shape::kGroups - 1) / Shape::kGroups;
  const int64_t fit = 228 * 1024 / static_cast<int64_t>(Shape::kSmem + 2048);   // 1 KB reserved per CTA, 1 KB static
  const int64_t most = int64_t{sms} * (fit < Shape::kMinBlocks ? fit : Shape::kMinBlocks);
  return want < most ? want : most;
}

template <int kT>
int launch_fwd(const NormParams& p, cudaStream_t s) {
  constexpr int kGroups = kBlockThreads<kT> / kT;
  const int64_t blocks = (p.N + kGroups - 1) / kGroups;
  block_norm_kernel<kT><<<static_cast<unsigned>(blocks), kBlockThreads<kT>, 0, s>>>(p);
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

// The partials of dw, one per CTA of the widest grid any device gets.
extern "C" size_t tpk_block_norm_bwd_workspace_bytes(int64_t N, int32_t C) {
  using namespace tpk;
  if (N < 0 || C < 8 || C % 8 || C > kMaxC) return 0;
  return bwd_shape(C, [&](auto shape, auto, auto) {
    return static_cast<size_t>(bwd_blocks<decltype(shape)>(N, kMaxSms)) * 2 * static_cast<size_t>(C) * 4;
  });
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
  int64_t blocks = 0;
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
    st = bwd_shape(C, [&](auto shape, auto kt, auto kv) {
      using Shape = decltype(shape);
      constexpr auto kern = block_norm_bwd_kernel<decltype(kt)::value, decltype(kv)::value>;
      static PerContext<int> rec;
      const int e = guarded([&] { return set_smem_once(rec, kern, Shape::kSmem); });
      if (e != TPK_OK) return e;
      blocks = bwd_blocks<Shape>(N, sms);
      kern<<<static_cast<unsigned>(blocks), Shape::kBlock, Shape::kSmem, s>>>(p);
      return cuda_status(cudaGetLastError());
    });
    if (st != TPK_OK) return st;
  }
  norm_dw_kernel<<<dim3((C + 31) / 32, 2), 1024, 0, s>>>(static_cast<const float*>(workspace),
                                                         static_cast<int>(blocks), C, dw_post, dw_pre);
  return cuda_status(cudaGetLastError());
}
