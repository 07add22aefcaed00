// Launchers of the kernels that train the experts in 16 bits: rows to the experts and back, the
// grouped product and its gradients, and the routing weights' gradient.
#pragma once

#include "mx.hpp"

namespace moe {

// ---- rows to the experts and back ----------------------------------------------------------
struct DispatchArgs {
  const void* x;
  int dtype;
  int64_t ldx;
  int T, H, K, rows;
  const int32_t* src;
  void* out;
  int64_t ldo;
};
hipError_t launch_dispatch_rows(const DispatchArgs& a, hipStream_t s);

struct CombineArgs {
  const void* rows;
  int dtype;
  int64_t ldr;
  int n_rows;
  const int32_t* slot;
  const float* w;        // nullptr: 1
  int T, K, H;
  const void* residual;  // of out's type, or nullptr
  int64_t ldres;
  void* out;
  int out_dtype;
  int64_t ldo;
};
hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t s);

struct CombineBackwardArgs {
  const void* grad_out;
  int grad_dtype;
  int64_t ldg;
  const int32_t* slot;
  const float* w;     // nullptr: 1
  int T, K, H, n_rows;
  const void* rows;   // with grad_w
  int dtype;
  int64_t ldr;
  void* grad_rows;    // or nullptr
  int64_t ldgr;
  float* grad_w;      // or nullptr
};
hipError_t launch_combine_rows_backward(const CombineBackwardArgs& a, hipStream_t s);

// ---- the grouped product and its gradients -------------------------------------------------
enum MmOp { kMmForward = 0, kMmDgrad = 1, kMmWgrad = 2 };

// Forward: out[r, n] = act(sum_k a[a(r), k] w[e, n, k] + bias[e, n]) + residual[r, n].
// Dgrad: out[r, k] = sum_n grad[r, n] w[e, n, k], with z through the SwiGLU that made the input.
// Wgrad: out[e, n, k] = sum_r grad[r, n] a[a(r), k], bias_out[e, n] = sum_r grad[r, n].
struct MmProblem {
  int op, dtype, out_dtype;
  bool swiglu;
  const void* w;           // [E x n x k]; n = 2 n_out for the forward's SwiGLU
  const void* a;           // forward, wgrad: rows of k_in
  int64_t lda;
  const void* grad;        // dgrad, wgrad: [rows x n_out]
  int64_t ldg;
  const int32_t* src;      // row r reads a's row src[r] / K; nullptr: row r
  const int32_t* offsets;  // [E + 1]
  const void* bias;        // [E x n] or nullptr
  const void* residual;    // of out's type, or nullptr
  int64_t ldres;
  void* z;                 // forward: written, or nullptr; dgrad: read
  int64_t ldz;
  void* out;
  int64_t ldo;
  void* bias_out;          // wgrad: [E x n_out] of out's type, or nullptr
  int n_out, k_in, E, n_act, K, rows;
  int parts;               // wgrad: of each expert's rows, out and bias_out having [E x parts]
  Division by_k;           // by K (set by the launcher)
};
hipError_t launch_mm_forward(const MmProblem& p, hipStream_t s);
hipError_t launch_mm_dgrad(const MmProblem& p, hipStream_t s);
hipError_t launch_mm_wgrad(const MmProblem& p, void* ws, hipStream_t s);
size_t mm_wgrad_workspace(int rows, int n_out, int k_in, int E);

// ---- the routing weights' gradient ----------------------------------------------------------
hipError_t launch_route_backward(const int32_t* idx, const float* w, const float* grad_w, int T,
                                 int E, int K, bool accumulate, void* grad_logits, int dtype,
                                 int64_t ld, hipStream_t s);

}  // namespace moe
