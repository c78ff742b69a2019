// Projections: y = act(x w^T + bias) + residual, and the gradients
//   dz = dy act'(z), z = x w^T + bias,   dx = dz w,   dw = dz^T x,   db = sum of dz's rows.
// The products and their epilogues are product.cuh's; few rows go to few.cu.
// With an activation the backward forms z again: one more product, and nothing
// the width of z is kept from the forward (z kept in bf16 would put its rounding
// into db, an fp32 sum).  dz is rounded to bf16 for its two products, as every
// operand of the tensor cores is; db sums it before that rounding.
#include "few.cuh"

namespace tpk {
namespace product {
namespace {

constexpr int kSumThreads = 256;   // 32 lanes of 8 columns x 8 rows at a time
constexpr int kSumCols = 256;
constexpr int kSumMost = 64;       // partial rows left for the last pass

template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  static __device__ __forceinline__ void add(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    v[0] += lo16(q.x); v[1] += hi16(q.x); v[2] += lo16(q.y); v[3] += hi16(q.y);
    v[4] += lo16(q.z); v[5] += hi16(q.z); v[6] += lo16(q.w); v[7] += hi16(q.w);
  }
};
template <>
struct Eight<float> {
  static __device__ __forceinline__ void add(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
};

// out[b][c] = sum of the rows b * per .. of m: a CTA takes 256 columns of `per` rows.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) column_sum_kernel(const T* __restrict__ m, int64_t rows, int cols,
                                                                 int64_t ld, int64_t per, float* __restrict__ out,
                                                                 int early) {
  __shared__ float4 part[8][32][2];
  ptx::dependents_launch();
  if (!early) ptx::dependency_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * kSumCols + lane * 8;
  const int64_t lo = static_cast<int64_t>(blockIdx.y) * per, hi = lo + per < rows ? lo + per : rows;
  float v[8] = {};
  if (c < cols) {
#pragma unroll 8
    for (int64_t r = lo + w; r < hi; r += 8) Eight<T>::add(m + r * ld + c, v);
  }
  part[w][lane][0] = make_float4(v[0], v[1], v[2], v[3]);
  part[w][lane][1] = make_float4(v[4], v[5], v[6], v[7]);
  __syncthreads();
  if (w < 2 && c < cols) {
    float4 s = part[0][lane][w];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const float4 x = part[i][lane][w];
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    *reinterpret_cast<float4*>(out + static_cast<int64_t>(blockIdx.y) * cols + c + w * 4) = s;
  }
  if (early) ptx::dependency_wait();
}

// Row blocks of the first pass: enough CTAs for two per SM, 32 rows each or more.
int64_t sum_rows(int64_t rows, int64_t cols) {
  const int64_t across = (cols + kSumCols - 1) / kSumCols;
  int64_t blocks = (2 * kMaxSms + across - 1) / across;
  blocks = blocks < 1 ? 1 : blocks > kSumMost ? kSumMost : blocks;
  const int64_t per = (rows + blocks - 1) / blocks;
  return per < 32 ? 32 : per;
}
int64_t sum_blocks(int64_t rows, int64_t cols) {
  const int64_t per = sum_rows(rows, cols);
  return (rows + per - 1) / per;
}

// Needs nothing of the stream's last kernel (as a product's `early`).
template <typename T>
int column_sums(const T* m, int64_t rows, int64_t cols, int64_t ld, float* part, float* out, cudaStream_t s) {
  const unsigned across = static_cast<unsigned>((cols + kSumCols - 1) / kSumCols);
  const int64_t per = sum_rows(rows, cols), blocks = sum_blocks(rows, cols);
  const int n = static_cast<int>(cols);
  const int st = launch_kernel(column_sum_kernel<T>, dim3(across, static_cast<unsigned>(blocks)), kSumThreads, 0, 1, true,
                               s, m, rows, n, ld, per, blocks == 1 ? out : part, 1);
  if (st != TPK_OK || blocks == 1) return st;
  return launch_kernel(column_sum_kernel<float>, dim3(across), kSumThreads, 0, 1, true, s, static_cast<const float*>(part),
                       blocks, n, cols, blocks, out, 0);
}

// The sum of a split product's partial tiles, 8 columns per thread, and kLin's
// epilogue.  residual may be out.
__global__ void __launch_bounds__(256) join_kernel(const float* __restrict__ acc, int M, int N, int whole, int splits,
                                                   const float* __restrict__ bias, int act,
                                                   const __nv_bfloat16* residual, int64_t ld_res, __nv_bfloat16* out,
                                                   int64_t ld_out) {
  ptx::dependents_launch();
  ptx::dependency_wait();
  const int mt = (M + kTile - 1) / kTile, nt = (N + kTile - 1) / kTile, tail = mt * nt - whole;
  const int64_t step = static_cast<int64_t>(tail) * (kTile * kTile);
  const int64_t items = static_cast<int64_t>(tail) * (kTile * kTile / 8);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; it < items;
       it += static_cast<int64_t>(gridDim.x) * 256) {
    int m, n;
    place_of(mt, nt, whole + static_cast<int>(it / (kTile * kTile / 8)), m, n);
    const int64_t r = static_cast<int64_t>(m) * kTile + it / (kTile / 8) % kTile;
    const int col = n * kTile + static_cast<int>(it % (kTile / 8)) * 8;
    if (r >= M || col >= N) continue;
    const float* from = acc + it * 8;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(from + s * step));
      const float4 b = __ldcg(reinterpret_cast<const float4*>(from + s * step) + 1);
      x.x += a.x; x.y += a.y; x.z += a.z; x.w += a.w;
      y.x += b.x; y.y += b.y; y.z += b.z; y.w += b.w;
    }
    uint64_t v[4] = {ptx::f2(x.x, x.y), ptx::f2(x.z, x.w), ptx::f2(y.x, y.y), ptx::f2(y.z, y.w)};
    if (bias) {
      const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(bias + col));
      const ulonglong2 b = __ldg(reinterpret_cast<const ulonglong2*>(bias + col) + 1);
      v[0] = ptx::add2(v[0], a.x);
      v[1] = ptx::add2(v[1], a.y);
      v[2] = ptx::add2(v[2], b.x);
      v[3] = ptx::add2(v[3], b.y);
    }
    if (act != TPK_ACT_NONE)
      with_act(act, [&](auto t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_2<decltype(t)::value>(v[e]);
      });
    if (residual) {
      const uint4 q = *reinterpret_cast<const uint4*>(residual + r * ld_res + col);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = ptx::add2(v[e], ptx::f2(lo16(w[e]), hi16(w[e])));
    }
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo, hi;
      ptx::unf2(v[e], lo, hi);
      o[e] = ptx::pack_bf16x2(lo, hi);
    }
    *reinterpret_cast<uint4*>(out + r * ld_out + col) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

int join(const Params& p, const float* bias, int act, const Mat& residual, const Mat& out, cudaStream_t s) {
  const int64_t blocks = (tiles_of(p.M, p.N) - p.whole) * (kTile / 8), most = int64_t{num_sms()} * 16;
  return launch_kernel(join_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0, 1, true, s,
                       static_cast<const float*>(p.acc), p.M, p.N, p.whole, p.splits, bias, act,
                       static_cast<const __nv_bfloat16*>(residual.p), residual.ld,
                       static_cast<__nv_bfloat16*>(const_cast<void*>(out.p)), out.ld);
}

// The plans of tpk_linear's products: y and dz [N, O] over C, dx [N, C] over O, dw [O, C] over N.
Plan forward_plan(int64_t N, int64_t C, int64_t O) { return plan_of(N, O, C); }
Plan input_plan(int64_t N, int64_t C, int64_t O) { return plan_of(N, C, O); }
Plan weight_plan(int64_t N, int64_t C, int64_t O) { return plan_of(O, C, N); }
// (dz's epilogue has no joined form)
Plan dz_plan(int64_t N, int64_t C, int64_t O) { return plan_of(N, O, C, false); }

Params params(int64_t M, int64_t N, int64_t K, const Plan& plan, float* acc, int32_t* err) {
  Params p{};
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.narrow = plan.narrow;
  p.teams = plan.teams;
  p.whole = static_cast<int32_t>(plan.split.whole);
  p.splits = plan.split.splits;
  p.acc = acc;
  p.err = err;
  return p;
}
// Stages of the longest sum that a pair adds up.
int64_t longest_of(const Plan& p, int64_t K) {
  const int64_t k = (K + 63) / 64;
  return p.narrow ? (k + p.teams - 1) / p.teams : p.split.whole > 0 || p.split.splits == 1 ? k : k / p.split.splits + 1;
}
// The product as planned, in single accumulations where they are short enough.
template <int kMode>
int launch_plan(const Maps& m, const Params& p, const Plan& plan, bool after, cudaStream_t s) {
  if (p.narrow) return launch<kMode, true, true>(m, p, after, s);
  if constexpr (kMode == kDx || kMode == kDw)
    if (longest_of(plan, p.K) > kChunk) return launch<kMode, false>(m, p, after, s);
  return launch<kMode, true>(m, p, after, s);
}

struct LinearWork {
  __nv_bfloat16* dz = nullptr;
  float *sums = nullptr, *part = nullptr, *acc = nullptr, *acc_w = nullptr;
};
size_t carve(uint8_t* base, int64_t N, int64_t C, int64_t O, int32_t act, bool backward, LinearWork* w) {
  LinearWork o;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = base + at;
    at += (bytes + 1023) / 1024 * 1024;
    return p;
  };
  if (!backward) {
    if (N > kFewRows) o.acc = reinterpret_cast<float*>(take(acc_bytes(forward_plan(N, C, O))));
  } else {
    if (act != TPK_ACT_NONE) {
      o.dz = reinterpret_cast<__nv_bfloat16*>(take(static_cast<size_t>(N * own_stride(O)) * 2));
      o.sums = reinterpret_cast<float*>(take(static_cast<size_t>((N + 31) / 32) * O * 4));
    }
    o.part = reinterpret_cast<float*>(take(static_cast<size_t>(kSumMost) * O * 4));
    o.acc = reinterpret_cast<float*>(take(acc_bytes(input_plan(N, C, O))));
    o.acc_w = reinterpret_cast<float*>(take(acc_bytes(weight_plan(N, C, O))));
  }
  if (w) *w = o;
  return at;
}

bool sizes_ok(int64_t N, int64_t C, int64_t O) {
  return N >= 0 && N < (int64_t{1} << 31) - 8192 && C >= 8 && C % 8 == 0 && O >= 8 && O % 8 == 0 && O <= (1 << 20);
}
// tiles of every product are counted in 32 bits
bool tiles_ok(int64_t N, int64_t C, int64_t O) { return tiles_of(N, C > O ? C : O) < (int64_t{1} << 27); }
bool act_ok(int32_t act) { return act >= TPK_ACT_NONE && act <= TPK_ACT_GELU_TANH; }
bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld % 8 == 0; }

}  // namespace

int linear_product(const Mat& x, const Mat& w, const float* bias, int act, const Mat& residual, const Mat& y,
                   float* acc, bool after, int32_t* err, cudaStream_t s) {
  if (x.rows <= kFewRows) return few_linear(x, w, bias, act, residual, y, after, err, s);
  Maps m;
  int st = map_of(&m.a, x, kHalf);
  const Plan plan = forward_plan(x.rows, x.cols, w.rows);
  if (st == TPK_OK) st = map_of(&m.b, w, plan.narrow ? kHalf / 2 : kHalf);
  if (st == TPK_OK) st = map_of(&m.out, y, kHalf);
  if (st == TPK_OK && residual.p) st = map_of(&m.in, residual, kHalf);
  if (st != TPK_OK) return st;
  Params p = params(x.rows, w.rows, x.cols, plan, acc, err);
  p.bias = bias;
  p.act = act;
  p.has_in = residual.p != nullptr;
  p.in = static_cast<const uint16_t*>(residual.p);
  p.ld_in = residual.ld;
  p.out = static_cast<uint16_t*>(const_cast<void*>(y.p));
  p.ld_out = y.ld;
  st = launch_plan<kLin>(m, p, plan, after, s);
  return st == TPK_OK && p.splits > 1 ? join(p, bias, act, residual, y, s) : st;
}

int input_product(const Mat& dz, const Mat& w, const Mat& dx, float* acc, bool after, int32_t* err, cudaStream_t s,
                  Params* left) {
  Maps m;
  int st = map_of(&m.a, dz, kHalf);
  if (st == TPK_OK) st = map_of(&m.b, w, 64);
  if (st == TPK_OK) st = map_of(&m.out, dx, kHalf);
  if (st != TPK_OK) return st;
  const Plan plan = input_plan(dz.rows, w.cols, dz.cols);
  Params p = params(dz.rows, w.cols, dz.cols, plan, acc, err);
  p.late = 1;
  p.out = static_cast<uint16_t*>(const_cast<void*>(dx.p));
  p.ld_out = dx.ld;
  *left = p;
  return launch_plan<kDx>(m, p, plan, after, s);
}

int weight_product(const Mat& dz, const Mat& x, const Mat& dw, float* acc, const Params& before, int32_t* err,
                   cudaStream_t s, Params* left) {
  Maps m;
  int st = map_of(&m.a, dz, 64);
  if (st == TPK_OK) st = map_of(&m.b, x, 64);
  if (st == TPK_OK) st = map_of(&m.out, dw, kHalf);
  if (st != TPK_OK) return st;
  const Plan plan = weight_plan(dz.rows, x.cols, dz.cols);
  Params p = params(dz.cols, x.cols, dz.rows, plan, acc, err);
  p.early = (before.narrow ? shape_of<kDx, true>(before) : shape_of<kDx>(before)).units * before.teams < kPairs;
  p.out = static_cast<uint16_t*>(const_cast<void*>(dw.p));
  p.ld_out = dw.ld;
  *left = p;
  return launch_plan<kDw>(m, p, plan, true, s);
}

int grads_product(const Grad* g, int n, Params& p, bool after, int32_t* err, cudaStream_t s) {
  Maps m;
  CUtensorMap* const a[3] = {&m.a, &m.in, &m.more};
  CUtensorMap* const b[3] = {&m.b, &m.b2, &m.in2};
  CUtensorMap* const out[3] = {&m.out, &m.out2, &m.out3};
  int st = TPK_OK;
  bool taken[3] = {};
  for (int i = 0; i < n; ++i) {   // the product that p.sub[i] describes
    int j = 0;
    while (taken[j] || g[j].out.rows != p.sub[i].M || g[j].out.cols != p.sub[i].N || g[j].amn != (p.sub[i].amn != 0)) ++j;
    taken[j] = true;
    if (st == TPK_OK) st = map_of(a[i], g[j].a, g[j].amn ? 64 : kHalf);
    if (st == TPK_OK) st = map_of(b[i], g[j].b, 64);
    if (st == TPK_OK) st = map_of(out[i], g[j].out, kHalf);
  }
  if (st != TPK_OK) return st;
  p.teams = 1;
  p.narrow = 1;
  p.splits = 1;
  p.late = 1;
  p.err = err;
  return launch<kGrads, true, true>(m, p, after, s);
}

int join_left(const Params& left, const Mat& out, cudaStream_t s) {
  return left.splits > 1 ? join(left, nullptr, TPK_ACT_NONE, Mat{}, out, s) : TPK_OK;
}

}  // namespace product
}  // namespace tpk

extern "C" size_t tpk_linear_workspace_bytes(int64_t N, int32_t C, int32_t O, int32_t act, int32_t backward) {
  using namespace tpk::product;
  if (!sizes_ok(N, C, O) || !tiles_ok(N, C, O) || N == 0) return 0;
  return carve(nullptr, N, C, O, act, backward != 0, nullptr);
}

extern "C" int tpk_linear_plan(int64_t N, int32_t C, int32_t O, int32_t act, int32_t backward, tpk_product_plan* out) {
  using namespace tpk::product;
  if (!out || !sizes_ok(N, C, O) || !act_ok(act)) return TPK_E_ARG;
  if (C > kMostK) return TPK_E_UNSUPPORTED;
  if (!tiles_ok(N, C, O)) return TPK_E_OVERFLOW;
  if (N == 0) return 0;
  int n = 0;
  auto put = [&](int32_t product, const Plan& p, int64_t M, int64_t width, int64_t K, bool may_stop) {
    const int64_t longest = longest_of(p, K);
    out[n++] = tpk_product_plan{product, p.narrow ? TPK_FORM_NARROW : TPK_FORM_WIDE, p.teams,
                                static_cast<int32_t>(p.narrow ? p.split.whole : tiles_of(M, width)),
                                static_cast<int32_t>(p.split.tail), p.split.splits,
                                static_cast<int32_t>(may_stop ? (longest + kChunk - 1) / kChunk : 1)};
  };
  if (!backward) {
    if (N <= kFewRows)
      out[n++] = tpk_product_plan{TPK_PRODUCT_Y, TPK_FORM_FEW, 1, 0, 0, 1, 1};
    else
      put(TPK_PRODUCT_Y, forward_plan(N, C, O), N, O, C, false);
    return n;
  }
  if (act != TPK_ACT_NONE) put(TPK_PRODUCT_DZ, dz_plan(N, C, O), N, O, C, false);
  const Mat dz{nullptr, N, O, O}, w{nullptr, O, C, C}, x{nullptr, N, C, C};
  const Grad grads[2] = {{dz, false, w, x}, {dz, true, x, w}};
  Params both{};
  if (grads_plan(grads, 2, &both)) {
    for (int32_t product : {TPK_PRODUCT_DX, TPK_PRODUCT_DW}) {
      const Sub& s = both.sub[(both.sub[0].amn != 0) == (product == TPK_PRODUCT_DW) ? 0 : 1];
      out[n++] = tpk_product_plan{product, TPK_FORM_TOGETHER, 1, s.mt * s.nt, 0, 1, 1};
    }
    return n;
  }
  put(TPK_PRODUCT_DX, input_plan(N, C, O), N, C, O, true);
  put(TPK_PRODUCT_DW, weight_plan(N, C, O), O, C, N, true);
  return n;
}

extern "C" int tpk_linear(const void* x, int64_t ld_x, const void* w, const float* bias, int32_t act,
                          const void* residual, int64_t ld_res, void* y, int64_t ld_y, int64_t N, int32_t C, int32_t O,
                          void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream) {
  using namespace tpk;
  using namespace tpk::product;
  if (!sizes_ok(N, C, O) || !act_ok(act) || !ld_ok(ld_x, C) || !ld_ok(ld_y, O)) return TPK_E_ARG;
  if (residual && !ld_ok(ld_res, O)) return TPK_E_ARG;
  if (C > kMostK) return TPK_E_UNSUPPORTED;
  if (!tiles_ok(N, C, O)) return TPK_E_OVERFLOW;
  if (N == 0) return TPK_OK;
  if (!x || !w || !y || y == x || y == w || !aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(residual) || !aligned16(bias))
    return TPK_E_ARG;
  if (residual == y && ld_res != ld_y && N > 1) return TPK_E_ARG;
  LinearWork k;
  const size_t need = carve(static_cast<uint8_t*>(workspace), N, C, O, act, false, &k);
  if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || ws_bytes < need)) return TPK_E_WORKSPACE;
  const int st = check_device();
  if (st != TPK_OK) return st;
  return linear_product(Mat{x, N, C, ld_x}, Mat{w, O, C, C}, bias, act, Mat{residual, N, O, ld_res}, Mat{y, N, O, ld_y},
                        k.acc, false, dev_err, static_cast<cudaStream_t>(stream));
}

extern "C" int tpk_linear_bwd(const void* x, int64_t ld_x, const void* w, const float* bias, int32_t act,
                              const void* dy, int64_t ld_dy, void* dx, int64_t ld_dx, void* dw, float* db, int64_t N,
                              int32_t C, int32_t O, void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream) {
  using namespace tpk;
  using namespace tpk::product;
  if (!sizes_ok(N, C, O) || !act_ok(act) || !ld_ok(ld_x, C) || !ld_ok(ld_dy, O) || !ld_ok(ld_dx, C)) return TPK_E_ARG;
  if (C > kMostK) return TPK_E_UNSUPPORTED;
  if (!tiles_ok(N, C, O)) return TPK_E_OVERFLOW;
  if (!dw || !aligned16(dw) || !aligned16(db)) return TPK_E_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int st;
  if (N == 0) {
    st = check_device();
    if (st == TPK_OK) st = cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(O) * C * 2, s));
    if (st == TPK_OK && db) st = cuda_status(cudaMemsetAsync(db, 0, static_cast<size_t>(O) * 4, s));
    return st;
  }
  if (!x || !w || !dy || !dx || dx == x || dx == dy || dx == w || !aligned16(x) || !aligned16(w) || !aligned16(dy) || !aligned16(dx) || !aligned16(bias))
    return TPK_E_ARG;
  LinearWork k;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      ws_bytes < carve(static_cast<uint8_t*>(workspace), N, C, O, act, true, &k))
    return TPK_E_WORKSPACE;
  st = check_device();
  if (st != TPK_OK) return st;
  const Mat mx{x, N, C, ld_x}, mw{w, O, C, C};
  Mat dz{dy, N, O, ld_dy};
  if (act != TPK_ACT_NONE) {
    Maps m;
    st = map_of(&m.a, mx, kHalf);
    const Plan plan = dz_plan(N, C, O);
    Params p = params(N, O, C, plan, nullptr, dev_err);
    if (st == TPK_OK) st = map_of(&m.b, mw, p.narrow ? kHalf / 2 : kHalf);
    if (st == TPK_OK) st = map_of(&m.in, dz, kHalf);
    p.in = static_cast<const uint16_t*>(dy);
    p.ld_in = ld_dy;
    p.out = reinterpret_cast<uint16_t*>(k.dz);
    p.ld_out = own_stride(O);
    dz = Mat{k.dz, N, O, own_stride(O)};
    if (st == TPK_OK) st = map_of(&m.out, dz, kHalf);
    p.bias = bias;
    p.act = act;
    p.colsum = db ? k.sums : nullptr;
    if (st == TPK_OK) st = launch_plan<kDz>(m, p, plan, false, s);
  }
  const Mat mdx{dx, N, C, ld_dx}, mdw{dw, O, C, C};
  Params px{}, pw{}, both{};
  px.splits = pw.splits = 1;
  const Grad grads[2] = {{dz, false, mw, mdx}, {dz, true, mx, mdw}};
  if (grads_plan(grads, 2, &both)) {
    if (st == TPK_OK) st = grads_product(grads, 2, both, act != TPK_ACT_NONE, dev_err, s);
  } else {
    if (st == TPK_OK) st = input_product(dz, mw, mdx, k.acc, act != TPK_ACT_NONE, dev_err, s, &px);
    if (st == TPK_OK) st = weight_product(dz, mx, mdw, k.acc_w, px, dev_err, s, &pw);
  }
  if (st == TPK_OK && db)
    st = act != TPK_ACT_NONE
             ? column_sums(k.sums, (N + 31) / 32, O, O, k.part, db, s)
             : column_sums(static_cast<const __nv_bfloat16*>(dy), N, O, ld_dy, k.part, db, s);
  if (st == TPK_OK) st = join_left(px, mdx, s);
  if (st == TPK_OK) st = join_left(pw, mdw, s);
  return st;
}
