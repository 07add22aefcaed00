// C ABI of the MXFP4 operators, the bf16 combine and the balance loss: argument checks, then the
// launch.
#include <hip/hip_runtime.h>

#include "layout.hpp"
#include "moe_prefill.h"
#include "mx.hpp"

namespace {

using namespace moe;

static_assert((int)MOE_F32 == kF32 && (int)MOE_BF16 == kBF16 && (int)MOE_F16 == kF16,
              "the ABI's types");
static_assert(MOE_MX_F32 == kMxF32 && MOE_MX_BF16 == kMxBF16 && MOE_MX_SWIGLU_MXFP4 == kMxSwiglu,
              "the ABI's epilogues");

bool valid_dtype(int dt) { return dt >= MOE_F32 && dt <= MOE_F16; }
int64_t size_of(int dt) { return dt == MOE_F32 ? 4 : 2; }

constexpr long long kMaxRows = 1LL << 30;    // row indices are int32
constexpr long long kMaxGroups = 1LL << 23;  // workgroups of 512 threads or fewer in a grid's x

// rows of n values, ld apart, each 16-byte aligned (ld may be anything for a single row)
bool rows_ok(const void* p, int dt, int64_t ld, int rows, int64_t n) {
  if (!aligned(p, 16)) return false;
  return rows == 1 || (ld >= n && ld * size_of(dt) % 16 == 0);
}

int check_balance(const void* logits, int dtype, int64_t ld, int T, int E, int K) {
  if (!logits || T < 1 || E < 1 || K < 1 || K > E) return MOE_EINVAL;
  if (T > 1 && ld < E) return MOE_EINVAL;
  if (!valid_dtype(dtype) || E > MOE_MAX_E || K > MOE_MAX_K) return MOE_EUNSUPPORTED;
  if (!aligned(logits, (size_t)size_of(dtype))) return MOE_EINVAL;
  if ((long long)T * K > kMaxRows) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_mxfp4_quantize(const void* x, int dtype, int64_t ldx, int rows, int n, void* codes,
                       void* scales, void* stream) {
  if (!x || !codes || !scales || rows < 1 || n < 1) return MOE_EINVAL;
  if (!valid_dtype(dtype) || n % kMxBlock != 0) return MOE_EUNSUPPORTED;
  if (rows > kMaxRows) return MOE_EUNSUPPORTED;
  if (!rows_ok(x, dtype, ldx, rows, n) || !aligned(codes, 16)) return MOE_EINVAL;
  return status_of(launch_mx_quantize(x, dtype, rows == 1 ? n : ldx, rows, n,
                                      static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                                      as_stream(stream)));
}

int moe_mxfp4_dequantize(const void* codes, const void* scales, int rows, int n, void* y,
                         int dtype, int64_t ldy, void* stream) {
  if (!codes || !scales || !y || rows < 1 || n < 1) return MOE_EINVAL;
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || n % kMxBlock != 0) return MOE_EUNSUPPORTED;
  if (rows > kMaxRows) return MOE_EUNSUPPORTED;
  if (!rows_ok(y, dtype, ldy, rows, n) || !aligned(codes, 16)) return MOE_EINVAL;
  return status_of(launch_mx_dequantize(static_cast<const uint8_t*>(codes),
                                        static_cast<const uint8_t*>(scales), rows, n, y, dtype,
                                        rows == 1 ? n : ldy, as_stream(stream)));
}

int moe_mxfp4_mm_grouped(const void* w_codes, const void* w_scales, int n_out, int k_in,
                         const int32_t* offsets, int E, const void* a_codes, const void* a_scales,
                         int n_act, const int32_t* src, int K, int rows, int epilogue, void* out,
                         void* out_scales, void* stream) {
  if (!w_codes || !w_scales || !offsets || !a_codes || !a_scales || !out) return MOE_EINVAL;
  if (n_out < 1 || k_in < 1 || E < 1 || rows < 1 || n_act < 1 || (src && K < 1))
    return MOE_EINVAL;
  if (epilogue < MOE_MX_F32 || epilogue > MOE_MX_SWIGLU_MXFP4) return MOE_EINVAL;
  if (epilogue == MOE_MX_SWIGLU_MXFP4 && !out_scales) return MOE_EINVAL;
  if (!src && n_act < rows) return MOE_EINVAL;
  if (n_out % 32 != 0 || k_in % 128 != 0 || E > MOE_MAX_E) return MOE_EUNSUPPORTED;
  if (src && K > MOE_MAX_K) return MOE_EUNSUPPORTED;
  // tiles are numbered in 31 bits, a grid's y holds 16, and rows are addressed by 32-bit offsets
  // from an expert's matrix and from a_codes
  const int64_t mats = epilogue == MOE_MX_SWIGLU_MXFP4 ? 2 : 1;
  if (rows / 32 + E > kMaxGroups || n_out / 32 > 65535 ||
      ((int64_t)rows / 32 + E) * (n_out / 32) >= (int64_t)1 << 31 ||
      mats * n_out * (k_in / 2) >= (int64_t)1 << 32 ||
      (int64_t)n_act * (k_in / 2) >= (int64_t)1 << 32)
    return MOE_EUNSUPPORTED;
  if (!aligned(w_codes, 16) || !aligned(a_codes, 16) || !aligned(w_scales, 4) ||
      !aligned(a_scales, 4) || !aligned(out, 16))
    return MOE_EINVAL;
  MxProblem p{};
  p.w = static_cast<const uint8_t*>(w_codes);
  p.ws = static_cast<const uint8_t*>(w_scales);
  p.offsets = offsets;
  p.a = static_cast<const uint8_t*>(a_codes);
  p.as = static_cast<const uint8_t*>(a_scales);
  p.src = src;
  p.out = out;
  p.out_scales = static_cast<uint8_t*>(out_scales);
  p.n_out = n_out;
  p.k_in = k_in;
  p.E = E;
  p.n_act = n_act;
  p.K = src ? K : 1;
  p.rows = rows;
  p.epilogue = epilogue;
  return status_of(launch_mx_mm(p, as_stream(stream)));
}

int moe_combine_bf16(const void* rows, const int32_t* slot, const float* topk_w, int T, int K,
                     int H, float* out, void* stream) {
  if (!rows || !slot || !topk_w || !out || T < 1 || K < 1 || H < 1) return MOE_EINVAL;
  if (!aligned(rows, 16) || !aligned(out, 16)) return MOE_EINVAL;
  if (H % 8 != 0 || K > MOE_MAX_K || (long long)T * K > kMaxRows) return MOE_EUNSUPPORTED;
  if (T > kMaxGroups || H / 8 > 256 * 65535) return MOE_EUNSUPPORTED;
  return status_of(launch_combine_bf16(rows, slot, topk_w, T, K, H, out, as_stream(stream)));
}

size_t moe_balance_workspace_size(int T, int E) {
  if (T < 1 || T > kMaxRows || E < 1 || E > MOE_MAX_E) return 0;
  return (size_t)kBalanceHeader + (size_t)balance_groups(T) * E * 8;
}

int moe_balance_loss(const void* logits, int dtype, int64_t ld, int T, int E,
                     const int32_t* topk_idx, int K, const uint8_t* valid, int32_t* counts,
                     float* prob_mean, float* loss, void* ws, size_t ws_bytes, void* stream) {
  if (!topk_idx || !counts || !prob_mean || !loss || !ws) return MOE_EINVAL;
  const int rc = check_balance(logits, dtype, ld, T, E, K);
  if (rc != MOE_OK) return rc;
  if (!aligned(ws, 4)) return MOE_EINVAL;
  if (ws_bytes < moe_balance_workspace_size(T, E)) return MOE_EWORKSPACE;
  const BalanceArgs a{logits, dtype, ld, T, E, K, topk_idx, valid};
  return status_of(launch_balance_loss(a, counts, prob_mean, loss, ws, as_stream(stream)));
}

int moe_balance_loss_backward(const void* logits, int dtype, int64_t ld, int T, int E,
                              const int32_t* counts, int K, const uint8_t* valid,
                              const float* grad_loss, void* grad_logits, int64_t ld_grad,
                              void* stream) {
  if (!counts || !grad_logits) return MOE_EINVAL;
  const int rc = check_balance(logits, dtype, ld, T, E, K);
  if (rc != MOE_OK) return rc;
  if (T > 1 && ld_grad < E) return MOE_EINVAL;
  // in place a row's gradient may be written before another row is read
  if (T > 1 && grad_logits == logits && ld_grad != ld) return MOE_EINVAL;
  if (!aligned(grad_logits, (size_t)size_of(dtype))) return MOE_EINVAL;
  const BalanceArgs a{logits, dtype, ld, T, E, K, nullptr, valid};
  return status_of(launch_balance_backward(a, counts, grad_loss, grad_logits, ld_grad,
                                           as_stream(stream)));
}

}  // extern "C"
