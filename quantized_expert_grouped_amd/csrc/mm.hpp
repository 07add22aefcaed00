// What the grouped products' kernels share: 16-bit types and their matrix instruction, and what is
// done with four neighbouring results of one row.
#pragma once

#include "common.hpp"
#include "train.hpp"

namespace moe {

constexpr int kMaxExperts = 2048;  // MOE_MAX_E

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));

template <int DT>
struct Half {  // kBF16 or kF16
  typedef typename Elem<DT>::type T;
  typedef T v4 __attribute__((ext_vector_type(4)));
  typedef T v8 __attribute__((ext_vector_type(8)));
};

// D[i, j] += sum_k P[i, k] Q[j, k] over 16 k: lane l holds row l % 32 of P and of Q, k = 8 (l / 32)
// .. + 7, and of D column j = l % 32, rows i = 8 (q / 4) + 4 (l / 32) + q % 4 in register q.
template <int DT>
__device__ __forceinline__ v16f mfma16(const v4i& p, const v4i& q, const v16f& c) {
  typedef typename Half<DT>::v8 v8;
  const v8 a = __builtin_bit_cast(v8, p), b = __builtin_bit_cast(v8, q);
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ v4f load4(const void* p, int64_t at) {
  typedef typename Elem<DT>::type v4 __attribute__((ext_vector_type(4)));
  const v4 v = *reinterpret_cast<const v4*>(static_cast<const typename Elem<DT>::type*>(p) + at);
  return (v4f){(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t at, const v4f& y) {
  typedef typename Elem<DT>::type T;
  typedef T v4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<v4*>(static_cast<T*>(p) + at) = (v4){(T)y[0], (T)y[1], (T)y[2], (T)y[3]};
}

// 1 / (1 + e^-g) with the hardware's exponential and reciprocal, 1 ulp each; the roundings of the
// exponent's argument and of its constant add 1.25 |g| 2^-24.  The result goes into 16 bits.  From
// g = -87.4 down 1 + e is 2^126 or more, whose reciprocal the hardware takes for 0.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

// dg and du, the gradients of gate and up from that of h = g s(g) u, s the sigmoid:
//   dg = dh u s(g) (1 + g (1 - s(g))),   du = dh g s(g).
// dh s(g) comes first: dh u or dh g alone can leave fp32's range where the gradient is small, and an
// infinity gives NaN with s = 0.  (Where dh s is subnormal it is off by 2^-150 at most, dg by 2^-143 |u|:
// g is above -87.4 there, since s is 0 below.)
__device__ __forceinline__ void swiglu_gradient(const v4f& dh, const v4f& g, const v4f& u, v4f& dg,
                                                v4f& du) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float s = sigmoid(g[q]);
    const float ds = dh[q] * s;
    du[q] = ds * g[q];
    dg[q] = ds * u[q] * fmaf(g[q], 1.0f - s, 1.0f);
  }
}

// The row of a that a route reads; the nearest one for a route outside.
__device__ __forceinline__ int act_row(const MmProblem& p, int route) {
  return route_row(route, p.by_k.mul, p.by_k.shift, p.n_act);
}

// The lane's sum of v over the lanes up to it: within rows of 16 lanes, then over the rows.
__device__ __forceinline__ int lane_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

}  // namespace moe
