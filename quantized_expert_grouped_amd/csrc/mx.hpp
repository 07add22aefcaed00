// MXFP4 (32 e2m1 values to a power-of-two scale, "OCP Microscaling Formats (MX) Specification",
// section 6.3) on the device, the types that the entry points around it take, and the launchers of
// the kernels that read or write it, of the bf16 combine and of the balance loss.
//
// A block's scale byte is max(exponent field of amax - 2, 0), so the scale 2^(byte - 127) is
// 2^(floor(log2(amax)) - 2) wherever that is representable and amax / scale lies in [4, 8).  A
// value is v / scale, exact in fp32 (the product with a power of two), rounded to the nearest of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code, 6 beyond.  Byte 255 is NaN: a block that
// holds an infinity or a NaN gets it, with codes 0.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kMxBlock = 32;   // values per scale
enum MoeDtype { kF32 = 0, kBF16 = 1, kF16 = 2 };

template <int DT>
struct Elem;
template <>
struct Elem<kF32> {
  typedef float type;
};
template <>
struct Elem<kBF16> {
  typedef __bf16 type;
};
template <>
struct Elem<kF16> {
  typedef _Float16 type;
};

// The scale byte of a block with this largest magnitude.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
  const uint32_t ef = __float_as_uint(amax) >> 23 & 255u;
  return ef == 255u ? 255u : (ef > 2u ? ef - 2u : 0u);
}

// The larger magnitude of two or three values; a NaN among them gives NaN.
__device__ __forceinline__ float mx_amax(float m, float v) {
  return __builtin_elementwise_maximum(m, fabsf(v));
}

// The 8 codes (value i in nibble i) of 8 values of a block with this scale byte.
// v_cvt_scalef32_pk_fp4_f32 divides by the power of two that its scale operand's exponent field
// stands for (0: 2^-127), rounds to the nearest, ties to even, and gives 6 beyond 6; tested for
// every border and scale.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], uint32_t byte) {
  const float scale = __uint_as_float(byte << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  return byte == 255u ? 0u : w;
}

hipError_t launch_mx_quantize(const void* x, int dtype, int64_t ldx, int rows, int n,
                              uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int n,
                                void* y, int dtype, int64_t ldy, hipStream_t s);

struct MxProblem {
  const uint8_t* w;        // codes [E x n_mat x k_in / 2]
  const uint8_t* ws;       // scale bytes [E x n_mat x k_in / 32]
  const int32_t* offsets;  // [E + 1]
  const uint8_t* a;        // codes [n_act x k_in / 2]
  const uint8_t* as;       // scale bytes [n_act x k_in / 32]
  const int32_t* src;      // row r reads activation row src[r] / K; nullptr: row r
  void* out;
  uint8_t* out_scales;     // SwiGLU: the requantised rows' scale bytes
  int n_out;               // output columns
  int k_in, E, n_act, K, rows;
  uint32_t k_mul, k_shift;  // division by K (set by the launcher)
  int epilogue;            // kMxF32, kMxBF16, kMxSwiglu (n_mat = 2 n_out: gate, then up)
};
constexpr int kMxF32 = 0, kMxBF16 = 1, kMxSwiglu = 2;
hipError_t launch_mx_mm(const MxProblem& p, hipStream_t s);

hipError_t launch_combine_bf16(const void* rows, const int32_t* slot, const float* w, int T, int K,
                               int H, float* out, hipStream_t s);

// Balance loss: workgroups of the forward pass, each leaving one row of partial sums.
constexpr int kBalanceGroups = 256;
constexpr int kBalanceHeader = 2048;  // bytes of the workspace before those rows
inline int balance_groups(int T) {
  return T < 16 * kBalanceGroups ? (T + 15) / 16 : kBalanceGroups;
}
struct BalanceArgs {
  const void* logits;
  int dtype;
  int64_t ld;
  int T, E, K;
  const int32_t* idx;
  const uint8_t* valid;  // nullptr: every token
};
hipError_t launch_balance_loss(const BalanceArgs& a, int32_t* counts, float* prob_mean, float* loss,
                               void* ws, hipStream_t s);
hipError_t launch_balance_backward(const BalanceArgs& a, const int32_t* counts,
                                   const float* grad_loss, void* grad, int64_t ld_grad,
                                   hipStream_t s);

}  // namespace moe
