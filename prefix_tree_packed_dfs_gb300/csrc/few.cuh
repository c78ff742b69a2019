// A few rows through a projection, or through the gated half of a feed-forward
// block (the next tokens of running rollouts): see few.cu.
#pragma once
#include "product.cuh"

namespace tpk {
namespace product {

constexpr int kFewRows = TPK_FEW_ROWS;   // see few.cu

// y = act(x w^T + bias) + residual.  after: x (and residual) come from the
// stream's last kernel, which lets this one start early.
int few_linear(const Mat& x, const Mat& w, const float* bias, int act, const Mat& residual, const Mat& y, bool after,
               int32_t* err, cudaStream_t s);
// a = act(g) u, g = x w_gate^T, u = x w_up^T
int few_gate(const Mat& x, const Mat& w_gate, const Mat& w_up, int act, const Mat& a, int32_t* err, cudaStream_t s);

}  // namespace product
}  // namespace tpk
