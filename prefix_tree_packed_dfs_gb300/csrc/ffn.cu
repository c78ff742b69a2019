// The gated feed-forward block: g | u = x w_in^T (w_in [2 I, C], the gate's
// rows first), a = act(g) u, y = a w_out^T + residual, and its gradients
//   da = dy w_out,  dg = da u act'(g),  du = da act(g)
//   dx = (dg | du) w_in,  dw_in = (dg | du)^T x,  dw_out = dy^T a.
// Both input projections, the activation and the product are one kernel: a
// tile of the accumulator holds g and u of the same channels, and only a (and,
// for training, g and u) leaves it.  The backward's first kernel forms da and
// takes it straight to dg and du; da is never stored.
// a, dg and du are rounded to bf16, as operands of their products; g and u are
// kept for the backward as scaled fp16 (product.cuh).
#include "few.cuh"

namespace tpk {
namespace product {
namespace {

struct FfnWork {
  __nv_bfloat16 *a = nullptr, *dgu = nullptr;
  float *acc = nullptr, *acc_in = nullptr, *acc_out = nullptr;
};
size_t carve(uint8_t* base, int64_t N, int64_t C, int64_t I, int64_t O, bool backward, bool own_a, FfnWork* w) {
  FfnWork o;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = base + at;
    at += (bytes + 1023) / 1024 * 1024;
    return p;
  };
  if (!backward) {
    if (!own_a) o.a = reinterpret_cast<__nv_bfloat16*>(take(static_cast<size_t>(N * own_stride(I)) * 2));
    if (N > kFewRows) o.acc = reinterpret_cast<float*>(take(acc_bytes(N, O, I)));
  } else {
    o.dgu = reinterpret_cast<__nv_bfloat16*>(take(static_cast<size_t>(N * own_stride(2 * I)) * 2));
    o.acc = reinterpret_cast<float*>(take(acc_bytes(N, C, 2 * I)));
    o.acc_in = reinterpret_cast<float*>(take(acc_bytes(2 * I, C, N)));
    o.acc_out = reinterpret_cast<float*>(take(acc_bytes(O, I, N)));
  }
  if (w) *w = o;
  return at;
}

bool sizes_ok(int64_t N, int64_t C, int64_t I, int64_t O) {
  return N >= 0 && N < (int64_t{1} << 31) - 8192 && C >= 8 && C % 8 == 0 && I >= 8 && I % 8 == 0 && O >= 8 &&
         O % 8 == 0;
}
bool widths_ok(int64_t C, int64_t I, int64_t O) { return C <= kMostK && I <= kMostK && O <= kMostK; }
bool act_ok(int32_t act) { return act >= TPK_ACT_NONE && act <= TPK_ACT_GELU_TANH; }
bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld % 8 == 0; }
bool tiles_ok(int64_t N, int64_t C, int64_t I, int64_t O) {
  const int64_t wide = 2 * I > C ? 2 * I : C;
  return tiles_of(N, wide > O ? wide : O) < (int64_t{1} << 27);
}

Params params(int64_t M, int64_t N, int64_t K, int act, int32_t* err) {
  Params p{};
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.splits = 1;
  p.teams = 1;
  p.whole = INT32_MAX;   // nothing is split
  p.act = act;
  p.err = err;
  return p;
}

const __nv_bfloat16* bf(const void* p) { return static_cast<const __nv_bfloat16*>(p); }

// What the forward keeps: rows of g and u, 16 bits each, own_stride(I) apart, then the exponents.
struct Saved {
  Mat g, u;
  uint8_t* exps;
};
Saved saved_of(void* p, int64_t N, int64_t I) {
  const int64_t to_u = own_stride(I);
  return Saved{Mat{p, N, I, 2 * to_u}, Mat{bf(p) + to_u, N, I, 2 * to_u}, static_cast<uint8_t*>(p) + N * 4 * to_u};
}

}  // namespace
}  // namespace product
}  // namespace tpk

extern "C" size_t tpk_gated_ffn_workspace_bytes(int64_t N, int32_t C, int32_t I, int32_t O, int32_t backward) {
  using namespace tpk::product;
  if (!sizes_ok(N, C, I, O) || !widths_ok(C, I, O) || !tiles_ok(N, C, I, O) || N == 0) return 0;
  return carve(nullptr, N, C, I, O, backward != 0, false, nullptr);
}

extern "C" size_t tpk_gated_ffn_saved_bytes(int64_t N, int32_t I) {
  using namespace tpk::product;
  if (!sizes_ok(N, 8, I, 8) || I > kMostK) return 0;
  return static_cast<size_t>(N * 4 * own_stride(I)) + exp_bytes(N, I);
}

extern "C" int tpk_gated_ffn(const void* x, int64_t ld_x, const void* w_in, const void* w_out, int32_t act,
                             const void* residual, int64_t ld_res, void* saved, void* a, void* y, int64_t ld_y, int64_t N,
                             int32_t C, int32_t I, int32_t O, void* workspace, size_t ws_bytes, int32_t* dev_err,
                             void* stream) {
  using namespace tpk;
  using namespace tpk::product;
  if (!sizes_ok(N, C, I, O) || !act_ok(act) || !ld_ok(ld_x, C) || !ld_ok(ld_y, O)) return TPK_E_ARG;
  if (residual && !ld_ok(ld_res, O)) return TPK_E_ARG;
  if (!widths_ok(C, I, O)) return TPK_E_UNSUPPORTED;
  if (!tiles_ok(N, C, I, O)) return TPK_E_OVERFLOW;
  if (N == 0) return TPK_OK;
  if (!x || !w_in || !w_out || !y || y == x || !aligned16(x) || !aligned16(w_in) || !aligned16(w_out) || !aligned16(y) ||
      !aligned16(residual) || !aligned16(saved) || !aligned16(a))
    return TPK_E_ARG;
  if (residual == y && ld_res != ld_y && N > 1) return TPK_E_ARG;
  FfnWork k;
  const size_t need = carve(static_cast<uint8_t*>(workspace), N, C, I, O, false, a != nullptr, &k);
  if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || ws_bytes < need)) return TPK_E_WORKSPACE;
  int st = check_device();
  if (st != TPK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Mat mx{x, N, C, ld_x}, gate{w_in, I, C, C}, up{bf(w_in) + int64_t{I} * C, I, C, C}, down{w_out, O, I, I};
  const Mat ma{a ? a : k.a, N, I, a ? I : own_stride(I)}, res{residual, N, O, ld_res}, my{y, N, O, ld_y};
  if (N <= kFewRows && !saved) {
    st = few_gate(mx, gate, up, act, ma, dev_err, s);
    return st == TPK_OK ? few_linear(ma, down, nullptr, TPK_ACT_NONE, res, my, true, dev_err, s) : st;
  }
  Maps m;
  st = map_of(&m.a, mx, kHalf);
  if (st == TPK_OK) st = map_of(&m.b, gate, kHalf);
  if (st == TPK_OK) st = map_of(&m.b2, up, kHalf);
  if (st == TPK_OK) st = map_of(&m.out, ma, kHalf);
  const Saved k16 = saved_of(saved, N, I);
  if (st == TPK_OK && saved) st = map_of(&m.out2, k16.g, kHalf);
  if (st == TPK_OK && saved) st = map_of(&m.out3, k16.u, kHalf);
  if (st != TPK_OK) return st;
  Params p = params(N, I, C, act, dev_err);
  p.save = saved != nullptr;
  p.exps = k16.exps;
  p.exp_rows = exp_rows(N);
  st = launch<kGate, true>(m, p, false, s);
  return st == TPK_OK ? linear_product(ma, down, nullptr, TPK_ACT_NONE, res, my, k.acc, true, dev_err, s) : st;
}

extern "C" int tpk_gated_ffn_bwd(const void* x, int64_t ld_x, const void* w_in, const void* w_out, int32_t act,
                                 const void* dy, int64_t ld_dy, const void* saved, const void* a, void* dx, int64_t ld_dx,
                                 void* dw_in, void* dw_out, int64_t N, int32_t C, int32_t I, int32_t O, void* workspace,
                                 size_t ws_bytes, int32_t* dev_err, void* stream) {
  using namespace tpk;
  using namespace tpk::product;
  if (!sizes_ok(N, C, I, O) || !act_ok(act) || !ld_ok(ld_x, C) || !ld_ok(ld_dy, O) || !ld_ok(ld_dx, C))
    return TPK_E_ARG;
  if (!widths_ok(C, I, O)) return TPK_E_UNSUPPORTED;
  if (!tiles_ok(N, C, I, O)) return TPK_E_OVERFLOW;
  if (!dw_in || !dw_out || !aligned16(dw_in) || !aligned16(dw_out)) return TPK_E_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int st;
  if (N == 0) {
    st = check_device();
    if (st == TPK_OK) st = cuda_status(cudaMemsetAsync(dw_in, 0, static_cast<size_t>(4) * I * C, s));
    if (st == TPK_OK) st = cuda_status(cudaMemsetAsync(dw_out, 0, static_cast<size_t>(2) * O * I, s));
    return st;
  }
  if (!x || !w_in || !w_out || !dy || !saved || !a || !dx || dx == x || dx == dy || !aligned16(x) || !aligned16(w_in) || !aligned16(w_out) ||
      !aligned16(dy) || !aligned16(saved) || !aligned16(a) || !aligned16(dx))
    return TPK_E_ARG;
  FfnWork k;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      ws_bytes < carve(static_cast<uint8_t*>(workspace), N, C, I, O, true, true, &k))
    return TPK_E_WORKSPACE;
  st = check_device();
  if (st != TPK_OK) return st;
  const int64_t wide = 2 * int64_t{I};
  const Mat mx{x, N, C, ld_x}, mdy{dy, N, O, ld_dy};
  Maps m;
  st = map_of(&m.a, mdy, kHalf);
  if (st == TPK_OK) st = map_of(&m.b, Mat{w_out, O, I, I}, 64);
  const Saved k16 = saved_of(const_cast<void*>(saved), N, I);
  if (st == TPK_OK) st = map_of(&m.in, k16.g, kHalf);
  if (st == TPK_OK) st = map_of(&m.in2, k16.u, kHalf);
  const int64_t ld = own_stride(wide);
  if (st == TPK_OK) st = map_of(&m.out, Mat{k.dgu, N, I, ld}, kHalf);
  if (st == TPK_OK) st = map_of(&m.out2, Mat{k.dgu + I, N, I, ld}, kHalf);
  Params p = params(N, I, O, act, dev_err);
  p.exps = k16.exps;
  p.exp_rows = exp_rows(N);
  if (st == TPK_OK) st = launch<kGateBwd, true>(m, p, false, s);
  const Mat dgu{k.dgu, N, wide, ld};
  const Mat mdx{dx, N, C, ld_dx}, mdin{dw_in, wide, C, C}, mdout{dw_out, O, I, I};
  const Mat win{w_in, wide, C, C}, ma{a, N, I, I};
  const Grad grads[3] = {{dgu, false, win, mdx}, {dgu, true, mx, mdin}, {mdy, true, ma, mdout}};
  Params all{};
  if (grads_plan(grads, 3, &all)) return st == TPK_OK ? grads_product(grads, 3, all, true, dev_err, s) : st;
  Params px, pin, pout;
  if (st == TPK_OK) st = input_product(dgu, win, mdx, k.acc, true, dev_err, s, &px);
  if (st == TPK_OK) st = weight_product(dgu, mx, mdin, k.acc_in, px, dev_err, s, &pin);
  if (st == TPK_OK) st = weight_product(mdy, ma, mdout, k.acc_out, pin, dev_err, s, &pout);
  if (st == TPK_OK) st = join_left(px, mdx, s);
  if (st == TPK_OK) st = join_left(pin, mdin, s);
  if (st == TPK_OK) st = join_left(pout, mdout, s);
  return st;
}
