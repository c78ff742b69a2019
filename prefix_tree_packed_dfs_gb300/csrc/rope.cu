// RoPE at tree-depth positions ("DAG packing", section "Positions": the
// position id of a token is its depth, so every parent->child edge has
// relative distance 1 wherever the two tokens sit in the row).
//
// HBM-bound: each position's Q and K rows are read and written once.  A block
// takes kPosPerBlock positions; it first builds their d/2 (cos, sin) pairs in
// shared memory (shared by all heads of Q and K), then streams the rows with
// 16-byte accesses: a thread rotates 8 pairs (x_i, x_{i+d/2}).
// The angle depth * base^(-2i/d) is reduced to a fraction of a turn in fp64
// (exact for depths < 2^31), then evaluated with sincospif in fp32.
//
// rope_rows_kernel is the general form (tpk_rope_by_depth_ex): either pairing,
// a part of the head, any angle per position and pair, strided rows.
#include <cuda_bf16.h>

#include <cmath>

#include "rowwise.cuh"

namespace tpk {
namespace {

constexpr int kPosPerBlock = 4;
constexpr int kThreads = 256;

struct Turns {
  double v[64];   // base^(-2i/d) / (2 pi), i < d/2
};

__global__ void __launch_bounds__(kThreads) rope_kernel(const __nv_bfloat16* q_in, const __nv_bfloat16* k_in,
                                                        __nv_bfloat16* q_out, __nv_bfloat16* k_out,
                                                        const int32_t* __restrict__ depth, int64_t F, int Hq, int Hkv,
                                                        int D, Turns turns, int inverse) {
  __shared__ float cs[kPosPerBlock][64];
  __shared__ float sn[kPosPerBlock][64];
  const int half = D / 2;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * kPosPerBlock;
  for (int t = threadIdx.x; t < kPosPerBlock * half; t += blockDim.x) {
    const int p = t / half, i = t % half;
    const int64_t f = f0 + p;
    float c = 1.f, s = 0.f;
    if (f < F) {
      double x = static_cast<double>(__ldg(depth + f)) * turns.v[i];
      x -= rint(x);   // fraction of a turn in [-1/2, 1/2]
      sincospif(static_cast<float>(2.0 * x), &s, &c);
      if (inverse) s = -s;
    }
    cs[p][i] = c;
    sn[p][i] = s;
  }
  __syncthreads();
  const int chunks = D / 16;   // 8 pairs per chunk
  const int heads = Hq + Hkv;
  const int items = kPosPerBlock * heads * chunks;
  for (int it = threadIdx.x; it < items; it += blockDim.x) {
    const int p = it / (heads * chunks);
    const int rem = it % (heads * chunks);
    const int h = rem / chunks, c = rem % chunks;
    const int64_t f = f0 + p;
    if (f >= F) continue;
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    if (h < Hq) {
      src = q_in + (f * Hq + h) * D;
      dst = q_out + (f * Hq + h) * D;
    } else {
      src = k_in + (f * Hkv + (h - Hq)) * D;
      dst = k_out + (f * Hkv + (h - Hq)) * D;
    }
    const int i0 = c * 8;
    uint4 ua = *reinterpret_cast<const uint4*>(src + i0);
    uint4 ub = *reinterpret_cast<const uint4*>(src + half + i0);
    __nv_bfloat16* a = reinterpret_cast<__nv_bfloat16*>(&ua);
    __nv_bfloat16* b = reinterpret_cast<__nv_bfloat16*>(&ub);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = __bfloat162float(a[j]), y = __bfloat162float(b[j]);
      const float cc = cs[p][i0 + j], ss = sn[p][i0 + j];
      a[j] = __float2bfloat16_rn(x * cc - y * ss);
      b[j] = __float2bfloat16_rn(x * ss + y * cc);
    }
    *reinterpret_cast<uint4*>(dst + i0) = ua;
    *reinterpret_cast<uint4*>(dst + half + i0) = ub;
  }
}

// ---- the general form ---------------------------------------------------------
// Turns per position of each pair as a 64-bit fraction: the angle's place in its
// turn is the low 64 bits of an integer product, off by depth * 2^-65 at most,
// for any int32 depth.  (In fp64 the products and roundings alone would take a
// third of the kernel's time on this part.)
constexpr int kMostPairs = 128;      // rot <= 256
constexpr int kRowsMost = 16;        // positions per block
constexpr int kRowItems = 4;         // pieces per thread whose loads are in flight together

struct Fractions {
  uint64_t v[kMostPairs];
};

struct RopeRows {
  const __nv_bfloat16 *q_in, *k_in;
  __nv_bfloat16 *q_out, *k_out;
  int64_t ld_q, ld_k, ld_qo, ld_ko;
  const int32_t* depth;
  int64_t F;
  int32_t Hq, Hkv, D, rot;
  int32_t per;                       // positions per block
  uint32_t inv_pos, inv_head;        // 2^32 / pieces of a position, of a head, rounded up
  float factor, sign;
};

// a / b by the reciprocal inv = 2^32 / b, rounded up: exact while a * b < 2^32
// (a block's several positions are few pieces; a position has 2^16 heads of 64
// pieces at most).
__device__ __forceinline__ int quotient(int a, int b, uint32_t inv) {
  return b == 1 ? a : static_cast<int>(__umulhi(static_cast<uint32_t>(a), inv));
}

// The pairs' (cos, sin) of a position lie by twos, two of every piece side by
// side: neighbouring lanes, which hold neighbouring pieces, read neighbouring 16
// bytes.  (In the pairs' own order every read took four turns: rope_batch 196 us.)
// A piece is 16 bytes of a head, or, for a rotated piece of the half layout,
// the two whose channels make pairs.
template <bool kInter>
__global__ void __launch_bounds__(kThreads, 4) rope_rows_kernel(const RopeRows p, const Fractions fr) {
  __shared__ float4 cs[kRowsMost * kMostPairs / 2];
  constexpr int kPer = kInter ? 4 : 8;                         // pairs of a piece
  const int pairs = p.rot / 2;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * p.per;
  const int n = p.F - f0 < p.per ? static_cast<int>(p.F - f0) : p.per;
  const int turned = kInter ? p.rot / 8 : p.rot / 16;          // rotated pieces of a head
  const int per_head = turned + (p.D - p.rot) / 8;
  const int heads = p.Hq + p.Hkv, per_pos = heads * per_head;
  const int items = n * per_pos;
  for (int i0 = threadIdx.x; i0 - static_cast<int>(threadIdx.x) < items; i0 += kThreads * kRowItems) {
    uint4 a[kRowItems], b[kRowItems];
    int at[kRowItems];               // position * 256 + piece; -1: none
    __nv_bfloat16* dst[kRowItems];
#pragma unroll
    for (int j = 0; j < kRowItems; ++j) {
      const int it = i0 + j * kThreads;
      at[j] = -1;
      if (it >= items) continue;
      const int pos = p.per == 1 ? 0 : quotient(it, per_pos, p.inv_pos), rem = it - pos * per_pos;
      const int h = quotient(rem, per_head, p.inv_head), c = rem - h * per_head;
      const int64_t f = f0 + pos;
      const __nv_bfloat16* src;
      if (h < p.Hq) {
        src = p.q_in + f * p.ld_q + h * p.D;
        dst[j] = p.q_out + f * p.ld_qo + h * p.D;
      } else {
        src = p.k_in + f * p.ld_k + (h - p.Hq) * p.D;
        dst[j] = p.k_out + f * p.ld_ko + (h - p.Hq) * p.D;
      }
      at[j] = pos * 256 + c;
      const int ch = c < turned ? c * 8 : p.rot + (c - turned) * 8;
      a[j] = *reinterpret_cast<const uint4*>(src + ch);
      if (!kInter && c < turned) b[j] = *reinterpret_cast<const uint4*>(src + pairs + ch);
      dst[j] += ch;
    }
    if (i0 == static_cast<int>(threadIdx.x)) {   // the angles, while the first pieces are on their way
      for (int t = threadIdx.x; t < n * pairs; t += kThreads) {
        const int pos = t / pairs, i = t - pos * pairs;
        const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(__ldg(p.depth + f0 + pos))) * fr.v[i];
        float s, c;
        sincospif(static_cast<float>(static_cast<int64_t>(turn)) * 0x1p-63f, &s, &c);
        const int j = i % kPer;
        reinterpret_cast<float2*>(cs)[2 * (pos * (pairs / 2) + j / 2 * turned + i / kPer) + j % 2] =
            make_float2(c * p.factor, s * p.factor * p.sign);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kRowItems; ++j) {
      if (at[j] < 0) continue;
      const int pos = at[j] >> 8, c = at[j] & 255;
      if (c < turned) {
        uint32_t x[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
        const float4* at_c = cs + pos * (pairs / 2) + c;
        if constexpr (kInter) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float4 w = at_c[e / 2 * turned];
            const float u0 = lo16(x[e]), v0 = hi16(x[e]), u1 = lo16(x[e + 1]), v1 = hi16(x[e + 1]);
            x[e] = pack2(u0 * w.x - v0 * w.y, u0 * w.y + v0 * w.x);
            x[e + 1] = pack2(u1 * w.z - v1 * w.w, u1 * w.w + v1 * w.z);
          }
        } else {
          uint32_t y[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 w = at_c[e * turned];
            const float u0 = lo16(x[e]), u1 = hi16(x[e]), v0 = lo16(y[e]), v1 = hi16(y[e]);
            x[e] = pack2(u0 * w.x - v0 * w.y, u1 * w.z - v1 * w.w);
            y[e] = pack2(u0 * w.y + v0 * w.x, u1 * w.w + v1 * w.z);
          }
          *reinterpret_cast<uint4*>(dst[j] + pairs) = make_uint4(y[0], y[1], y[2], y[3]);
        }
        a[j] = make_uint4(x[0], x[1], x[2], x[3]);
      }
      *reinterpret_cast<uint4*>(dst[j]) = a[j];
    }
  }
}

}  // namespace
}  // namespace tpk

extern "C" int tpk_rope_by_depth(const void* q_in, const void* k_in, void* q_out, void* k_out,
                                 const int32_t* depth, int64_t F, int32_t Hq, int32_t Hkv, int32_t d, double base,
                                 int32_t inverse, void* stream) {
  using namespace tpk;
  if (F < 0 || !depth || (d != 64 && d != 128) || Hq < 0 || Hkv < 0 || !(base > 1.0)) return TPK_E_ARG;
  if ((q_in == nullptr) != (q_out == nullptr) || (k_in == nullptr) != (k_out == nullptr)) return TPK_E_ARG;
  if ((q_in && Hq <= 0) || (k_in && Hkv <= 0)) return TPK_E_ARG;
  if ((reinterpret_cast<uintptr_t>(q_in) | reinterpret_cast<uintptr_t>(k_in) | reinterpret_cast<uintptr_t>(q_out) |
       reinterpret_cast<uintptr_t>(k_out)) % 16)
    return TPK_E_ARG;
  if (F == 0 || (!q_in && !k_in)) return TPK_OK;
  int st = check_device();
  if (st != TPK_OK) return st;
  Turns turns;
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < d / 2; ++i) turns.v[i] = pow(base, -2.0 * i / d) / two_pi;
  const int64_t blocks = (F + kPosPerBlock - 1) / kPosPerBlock;
  if (blocks > 0x7fffffff) return TPK_E_OVERFLOW;
  rope_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16*>(q_in), static_cast<const __nv_bfloat16*>(k_in),
      static_cast<__nv_bfloat16*>(q_out), static_cast<__nv_bfloat16*>(k_out), depth, F, q_in ? Hq : 0,
      k_in ? Hkv : 0, d, turns, inverse);
  return cuda_status(cudaGetLastError());
}

extern "C" int tpk_rope_by_depth_ex(const void* q_in, int64_t ld_q, const void* k_in, int64_t ld_k, void* q_out,
                                    int64_t ld_qo, void* k_out, int64_t ld_ko, const int32_t* depth, int64_t F,
                                    int32_t Hq, int32_t Hkv, int32_t d, const tpk_rope_opts* opts, int32_t inverse,
                                    void* stream) {
  using namespace tpk;
  if (F < 0 || Hq < 0 || Hkv < 0 || !opts || d < 16 || d > 512 || d % 8) return TPK_E_ARG;
  const int rot = opts->rot;
  if (rot < 16 || rot % 16 || rot > d || rot > 2 * kMostPairs || !opts->freqs || !std::isfinite(opts->factor) ||
      (opts->interleaved & ~1))
    return TPK_E_ARG;
  if ((q_in == nullptr) != (q_out == nullptr) || (k_in == nullptr) != (k_out == nullptr)) return TPK_E_ARG;
  if ((q_in && Hq <= 0) || (k_in && Hkv <= 0)) return TPK_E_ARG;
  if (!aligned16(q_in) || !aligned16(k_in) || !aligned16(q_out) || !aligned16(k_out)) return TPK_E_ARG;
  const int64_t wq = int64_t{Hq} * d, wk = int64_t{Hkv} * d;
  if (q_in && (ld_q < wq || ld_qo < wq || ld_q % 8 || ld_qo % 8)) return TPK_E_ARG;
  if (k_in && (ld_k < wk || ld_ko < wk || ld_k % 8 || ld_ko % 8)) return TPK_E_ARG;
  if ((q_in && q_in == q_out && ld_q != ld_qo) || (k_in && k_in == k_out && ld_k != ld_ko)) return TPK_E_ARG;
  Fractions fr{};
  for (int i = 0; i < rot / 2; ++i) {
    if (!std::isfinite(opts->freqs[i])) return TPK_E_ARG;
    const double turns = opts->freqs[i] / 6.283185307179586476925286766559;
    double frac = turns - std::floor(turns);          // whole turns per position turn nothing
    if (frac >= 1.0) frac = 0.0;
    // 64 bits of the fraction, 32 at a time (each step exact)
    const double hi = std::floor(frac * 4294967296.0), lo = (frac * 4294967296.0 - hi) * 4294967296.0;
    fr.v[i] = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo + 0.5);
  }
  if (F == 0 || (!q_in && !k_in)) return TPK_OK;
  if (!depth) return TPK_E_ARG;
  if ((q_in ? Hq : 0) + int64_t{k_in ? Hkv : 0} > 65536) return TPK_E_UNSUPPORTED;
  const int st = check_device();
  if (st != TPK_OK) return st;
  RopeRows p{};
  p.q_in = static_cast<const __nv_bfloat16*>(q_in);
  p.k_in = static_cast<const __nv_bfloat16*>(k_in);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.ld_q = ld_q;
  p.ld_k = ld_k;
  p.ld_qo = ld_qo;
  p.ld_ko = ld_ko;
  p.depth = depth;
  p.F = F;
  p.Hq = q_in ? Hq : 0;
  p.Hkv = k_in ? Hkv : 0;
  p.D = d;
  p.rot = rot;
  p.factor = static_cast<float>(opts->factor);
  p.sign = inverse ? -1.f : 1.f;
  // as many positions as give every thread its pieces once
  const bool inter = opts->interleaved != 0;
  const int64_t per_pos = int64_t{p.Hq + p.Hkv} * ((inter ? rot / 8 : rot / 16) + (d - rot) / 8);
  int64_t per = kThreads * kRowItems / per_pos;
  p.per = static_cast<int32_t>(per < 1 ? 1 : per > kRowsMost ? kRowsMost : per);
  const int64_t per_head = (inter ? rot / 8 : rot / 16) + (d - rot) / 8;
  p.inv_pos = static_cast<uint32_t>(((int64_t{1} << 32) + per_pos - 1) / per_pos);
  p.inv_head = static_cast<uint32_t>(((int64_t{1} << 32) + per_head - 1) / per_head);
  const int64_t blocks = (F + p.per - 1) / p.per;
  if (blocks > 0x7fffffff) return TPK_E_OVERFLOW;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (inter)
    rope_rows_kernel<true><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p, fr);
  else
    rope_rows_kernel<false><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p, fr);
  return cuda_status(cudaGetLastError());
}
