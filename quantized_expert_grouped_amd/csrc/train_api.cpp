// C ABI of the 16-bit experts' training operators: argument checks, then the launch.
#include <hip/hip_runtime.h>

#include "layout.hpp"
#include "moe_prefill.h"
#include "train.hpp"

namespace {

using namespace moe;

constexpr long long kMaxRows = 1LL << 30;  // row and route numbers are int32
constexpr int kMaxGroups = 1 << 23;         // workgroups of 512 threads or fewer in a grid's x
constexpr long long kMaxBytes = 1LL << 31; // of what a kernel addresses by 32-bit offsets

bool valid_dtype(int dt) { return dt >= MOE_F32 && dt <= MOE_F16; }
bool half_dtype(int dt) { return dt == MOE_BF16 || dt == MOE_F16; }
int64_t size_of(int dt) { return dt == MOE_F32 ? 4 : 2; }

// rows of n values, ld apart (ld may be anything for a single row), at any element
bool matrix_ok(const void* p, int dt, int64_t ld, int rows, int64_t n) {
  return aligned(p, (size_t)size_of(dt)) && (rows == 1 || ld >= n);
}
// each 16-byte aligned
bool wide_ok(const void* p, int dt, int64_t ld, int rows, int64_t n) {
  return aligned(p, 16) && (rows == 1 || (ld >= n && ld * size_of(dt) % 16 == 0));
}

// what the grouped products' three calls share
int check_mm(int dtype, int out_dtype, int n_out, int k_in, int E, int rows, int64_t mat_rows) {
  if (n_out < 1 || k_in < 1 || E < 1 || rows < 1) return MOE_EINVAL;
  if (!half_dtype(dtype) || (out_dtype != dtype && out_dtype != MOE_F32)) return MOE_EUNSUPPORTED;
  if (n_out % 8 != 0 || k_in % 8 != 0 || E > MOE_MAX_E || rows > kMaxRows) return MOE_EUNSUPPORTED;
  // tiles are numbered in 31 bits
  const int64_t nt = n_out / 64 + 1, kt = k_in / 64 + 1;
  if (((int64_t)rows / 128 + E) * (nt > kt ? nt : kt) >= 1LL << 31 || E * nt * kt >= 1LL << 31)
    return MOE_EUNSUPPORTED;
  if (n_out >= 1 << 21 || k_in >= 1 << 21 || mat_rows * k_in * 2 >= kMaxBytes) return MOE_EUNSUPPORTED;
  return MOE_OK;
}
// activations read through src
int check_src(const int32_t* src, int K, int n_act, int rows, int64_t ld, int n) {
  if (n_act < 1 || (src ? K < 1 : n_act < rows)) return MOE_EINVAL;
  if (src && (K > MOE_MAX_K || ((n_act - 1) * ld + n) * 2 >= kMaxBytes)) return MOE_EUNSUPPORTED;
  return MOE_OK;
}
// strides of the rows that a tile addresses from its first
bool stride_fits(int64_t ld, int rows) { return rows == 1 || ld < kMaxBytes / 1024; }

}  // namespace

extern "C" {

int moe_dispatch_rows(const void* x, int dtype, int64_t ldx, int T, int H, const int32_t* src,
                      int K, int rows, void* out, int64_t ldo, void* stream) {
  if (!x || !src || !out || T < 1 || H < 1 || K < 1 || rows < 1) return MOE_EINVAL;
  if (!valid_dtype(dtype) || K > MOE_MAX_K) return MOE_EUNSUPPORTED;
  if ((long long)T * K > kMaxRows || rows > kMaxGroups) return MOE_EUNSUPPORTED;
  if (!matrix_ok(x, dtype, ldx, T, H) || !matrix_ok(out, dtype, ldo, rows, H)) return MOE_EINVAL;
  const DispatchArgs a{x, dtype, T == 1 ? H : ldx, T, H, K, rows, src, out, rows == 1 ? H : ldo};
  return status_of(launch_dispatch_rows(a, as_stream(stream)));
}

int moe_combine_rows(const void* rows, int dtype, int64_t ldr, int n_rows, const int32_t* slot,
                     const float* topk_w, int T, int K, int H, const void* residual, int64_t ldres,
                     void* out, int out_dtype, int64_t ldo, void* stream) {
  if (!rows || !slot || !out || n_rows < 1 || T < 1 || K < 1 || H < 1) return MOE_EINVAL;
  if (!valid_dtype(dtype) || (out_dtype != dtype && out_dtype != MOE_F32)) return MOE_EUNSUPPORTED;
  if (K > MOE_MAX_K || (long long)T * K > kMaxRows || n_rows > kMaxRows || T > kMaxGroups)
    return MOE_EUNSUPPORTED;
  if (!matrix_ok(rows, dtype, ldr, n_rows, H) || !matrix_ok(out, out_dtype, ldo, T, H))
    return MOE_EINVAL;
  if (residual && !matrix_ok(residual, out_dtype, ldres, T, H)) return MOE_EINVAL;
  // in place a row may be written before another is read
  if (residual == out && T > 1 && ldres != ldo) return MOE_EINVAL;
  const CombineArgs a{rows, dtype, n_rows == 1 ? H : ldr, n_rows, slot, topk_w, T, K, H, residual,
                      T == 1 ? H : ldres, out, out_dtype, T == 1 ? H : ldo};
  return status_of(launch_combine_rows(a, as_stream(stream)));
}

int moe_combine_rows_backward(const void* grad_out, int grad_dtype, int64_t ldg,
                              const int32_t* slot, const float* topk_w, int T, int K, int H,
                              int n_rows, const void* rows, int dtype, int64_t ldr,
                              void* grad_rows, int64_t ldgr, float* grad_w, void* stream) {
  if (!grad_out || !slot || T < 1 || K < 1 || H < 1 || n_rows < 1) return MOE_EINVAL;
  if ((!grad_rows && !grad_w) || (grad_w && !rows)) return MOE_EINVAL;
  if (!valid_dtype(dtype) || (grad_dtype != dtype && grad_dtype != MOE_F32))
    return MOE_EUNSUPPORTED;
  if (K > MOE_MAX_K || (long long)T * K > kMaxRows || n_rows > kMaxRows || T > kMaxGroups)
    return MOE_EUNSUPPORTED;
  if (!matrix_ok(grad_out, grad_dtype, ldg, T, H)) return MOE_EINVAL;
  if (grad_w && !matrix_ok(rows, dtype, ldr, n_rows, H)) return MOE_EINVAL;
  if (grad_rows && !matrix_ok(grad_rows, dtype, ldgr, n_rows, H)) return MOE_EINVAL;
  if (grad_w && grad_rows == rows && n_rows > 1 && ldgr != ldr) return MOE_EINVAL;
  const CombineBackwardArgs a{grad_out, grad_dtype, T == 1 ? H : ldg, slot, topk_w, T, K, H, n_rows,
                              rows, dtype, n_rows == 1 ? H : ldr, grad_rows,
                              n_rows == 1 ? H : ldgr, grad_w};
  return status_of(launch_combine_rows_backward(a, as_stream(stream)));
}

int moe_mm_grouped(const void* w, int dtype, int n_out, int k_in, const int32_t* offsets, int E,
                   const void* a, int64_t lda, int n_act, const int32_t* src, int K, int rows,
                   const void* bias, int activation, const void* residual, int64_t ldres, void* z,
                   int64_t ldz, void* out, int out_dtype, int64_t ldo, void* stream) {
  if (!w || !offsets || !a || !out) return MOE_EINVAL;
  if (activation != MOE_ACT_NONE && activation != MOE_ACT_SWIGLU) return MOE_EINVAL;
  const bool swiglu = activation == MOE_ACT_SWIGLU;
  int rc = check_mm(dtype, out_dtype, n_out, k_in, E, rows, swiglu ? 2LL * n_out : n_out);
  if (rc != MOE_OK) return rc;
  if (swiglu ? residual != nullptr : z != nullptr) return MOE_EINVAL;
  if (swiglu && out_dtype != dtype) return MOE_EUNSUPPORTED;
  if ((rc = check_src(src, K, n_act, rows, n_act == 1 ? k_in : lda, k_in)) != MOE_OK) return rc;
  if (!aligned(w, 16) || !wide_ok(a, dtype, lda, n_act, k_in) || (bias && !aligned(bias, 16)) ||
      (residual && !wide_ok(residual, out_dtype, ldres, rows, n_out)) ||
      (z && !wide_ok(z, dtype, ldz, rows, 2LL * n_out)) ||
      !wide_ok(out, out_dtype, ldo, rows, n_out))
    return MOE_EINVAL;
  if (residual == out && rows > 1 && ldres != ldo) return MOE_EINVAL;
  if (!stride_fits(lda, n_act)) return MOE_EUNSUPPORTED;
  MmProblem p{};
  p.op = kMmForward, p.dtype = dtype, p.out_dtype = out_dtype, p.swiglu = swiglu;
  p.w = w, p.a = a, p.lda = n_act == 1 ? k_in : lda, p.src = src, p.offsets = offsets;
  p.bias = bias, p.residual = residual, p.ldres = rows == 1 ? n_out : ldres;
  p.z = z, p.ldz = rows == 1 ? 2LL * n_out : ldz;
  p.out = out, p.ldo = rows == 1 ? n_out : ldo;
  p.n_out = n_out, p.k_in = k_in, p.E = E, p.n_act = n_act, p.K = src ? K : 1, p.rows = rows;
  return status_of(launch_mm_forward(p, as_stream(stream)));
}

int moe_mm_grouped_dgrad(const void* w, int dtype, int n_out, int k_in, const int32_t* offsets,
                         int E, const void* grad, int64_t ldg, int rows, const void* z, int64_t ldz,
                         void* out, int out_dtype, int64_t ldo, void* stream) {
  if (!w || !offsets || !grad || !out) return MOE_EINVAL;
  const int rc = check_mm(dtype, out_dtype, n_out, k_in, E, rows, n_out);
  if (rc != MOE_OK) return rc;
  if (z && out_dtype != dtype) return MOE_EUNSUPPORTED;
  const int64_t cols = z ? 2LL * k_in : k_in;
  if (!aligned(w, 16) || !wide_ok(grad, dtype, ldg, rows, n_out) ||
      (z && !wide_ok(z, dtype, ldz, rows, cols)) || !wide_ok(out, out_dtype, ldo, rows, cols))
    return MOE_EINVAL;
  if (z == out && rows > 1 && ldz != ldo) return MOE_EINVAL;
  if (!stride_fits(ldg, rows)) return MOE_EUNSUPPORTED;
  MmProblem p{};
  p.op = kMmDgrad, p.dtype = dtype, p.out_dtype = out_dtype, p.swiglu = z != nullptr;
  p.w = w, p.grad = grad, p.ldg = rows == 1 ? n_out : ldg, p.offsets = offsets;
  p.z = const_cast<void*>(z), p.ldz = rows == 1 ? cols : ldz;
  p.out = out, p.ldo = rows == 1 ? cols : ldo;
  p.n_out = n_out, p.k_in = k_in, p.E = E, p.n_act = rows, p.K = 1, p.rows = rows;
  return status_of(launch_mm_dgrad(p, as_stream(stream)));
}

size_t moe_mm_grouped_wgrad_workspace_size(int rows, int n_out, int k_in, int E) {
  if (check_mm(MOE_BF16, MOE_BF16, n_out, k_in, E, rows, n_out) != MOE_OK) return 0;
  return mm_wgrad_workspace(rows, n_out, k_in, E);
}

int moe_mm_grouped_wgrad(const void* grad, int dtype, int64_t ldg, int n_out, const void* a,
                         int64_t lda, int k_in, int n_act, const int32_t* src, int K,
                         const int32_t* offsets, int E, int rows, void* grad_w, int out_dtype,
                         void* grad_bias, void* ws, size_t ws_bytes, void* stream) {
  if (!grad || !a || !offsets || !grad_w) return MOE_EINVAL;
  int rc = check_mm(dtype, out_dtype, n_out, k_in, E, rows, n_out);
  if (rc != MOE_OK) return rc;
  if ((rc = check_src(src, K, n_act, rows, n_act == 1 ? k_in : lda, k_in)) != MOE_OK) return rc;
  if (!wide_ok(grad, dtype, ldg, rows, n_out) || !wide_ok(a, dtype, lda, n_act, k_in) ||
      !aligned(grad_w, 16) || (grad_bias && !aligned(grad_bias, 16)))
    return MOE_EINVAL;
  if (!stride_fits(ldg, rows) || !stride_fits(lda, n_act)) return MOE_EUNSUPPORTED;
  const size_t need = mm_wgrad_workspace(rows, n_out, k_in, E);
  if (need && (!ws || !aligned(ws, 16))) return MOE_EINVAL;
  if (ws_bytes < need) return MOE_EWORKSPACE;
  MmProblem p{};
  p.op = kMmWgrad, p.dtype = dtype, p.out_dtype = out_dtype;
  p.a = a, p.lda = n_act == 1 ? k_in : lda, p.grad = grad, p.ldg = rows == 1 ? n_out : ldg;
  p.src = src, p.offsets = offsets, p.out = grad_w, p.bias_out = grad_bias;
  p.n_out = n_out, p.k_in = k_in, p.E = E, p.n_act = n_act, p.K = src ? K : 1, p.rows = rows;
  return status_of(launch_mm_wgrad(p, ws, as_stream(stream)));
}

int moe_route_topk_backward(const int32_t* topk_idx, const float* topk_w, const float* grad_w,
                            int T, int E, int K, int accumulate, void* grad_logits, int dtype,
                            int64_t ld, void* stream) {
  if (!topk_idx || !topk_w || !grad_w || !grad_logits || T < 1 || E < 1 || K < 1 || K > E)
    return MOE_EINVAL;
  if (!valid_dtype(dtype) || E > MOE_MAX_E || K > MOE_MAX_K || (long long)T * K > kMaxRows ||
      T > kMaxGroups)
    return MOE_EUNSUPPORTED;
  if (!matrix_ok(grad_logits, dtype, ld, T, E)) return MOE_EINVAL;
  return status_of(launch_route_backward(topk_idx, topk_w, grad_w, T, E, K, accumulate != 0,
                                         grad_logits, dtype, T == 1 ? E : ld, as_stream(stream)));
}

}  // extern "C"
