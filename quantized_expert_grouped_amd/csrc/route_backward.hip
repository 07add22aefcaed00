// The gradient of the router's logits.  The K routing weights are the softmax of the K chosen
// logits, so with gw = d loss / d w
//   d loss / d logits[t, idx[t, k]] = w_k (gw_k - sum_j w_j gw_j),
// and 0 for the other experts.  A route whose id is outside [0, E) has no expert row: w_k gw_k
// counts as 0, whatever the two are.  An id that comes twice gets the sum, in the order of k.
//
// G lanes to a token (16, 32 or 64, K of them with a route), so a wavefront holds 64 / G tokens.  It
// writes their rows' zeros, which need no input, in 16-byte pieces while the inputs come, waits for
// them, and writes the K values over them.  Bound by those writes (30118 x 512 bf16, 31 MB: 9.3 us).
#include "common.hpp"
#include "train.hpp"

namespace moe {

namespace {

constexpr int kWaves = 4;

template <int DT, int G>
__global__ __launch_bounds__(kWaves * 64) void route_backward_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ w, const float* __restrict__ grad_w,
    int T, int E, int K, bool accumulate, void* grad_logits, int64_t ld) {
  typedef typename Elem<DT>::type V;
  constexpr int kVec = 16 / sizeof(V);
  typedef V vec __attribute__((ext_vector_type(kVec), aligned(sizeof(V))));
  const int lane = threadIdx.x & 63;
  const int t0 = (blockIdx.x * kWaves + (threadIdx.x >> 6)) * (64 / G);
  const int t = t0 + lane / G, k = lane % G;
  const bool there = t < T && k < K;
  int id = -1;
  float wk = 0.0f, gw = 0.0f;
  if (there) {
    const int64_t at = (int64_t)t * K + k;
    id = idx[at];
    wk = w[at];
    gw = grad_w[at];
  }
  V* const grad = static_cast<V*>(grad_logits);
  if (!accumulate) {
    const vec zero = {};
    const int pieces = E / kVec;
    for (int x = 0; x < 64 / G && t0 + x < T; ++x) {
      V* row = grad + (int64_t)(t0 + x) * ld;
      for (int c = lane; c < pieces; c += 64) *reinterpret_cast<vec*>(row + c * kVec) = zero;
      const int c = pieces * kVec + lane;
      if (c < E) row[c] = (V)0.0f;
    }
  }
  const bool on = there && id >= 0 && id < E;
  if (!on) gw = wk = 0.0f;
  float sum = wk * gw;
#pragma unroll
  for (int o = G / 2; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  const float d = on ? wk * (gw - sum) : 0.0f;
  float all = 0.0f;  // of the routes with this id
  for (int j = 0; j < K; ++j) {
    const int from = (lane & ~(G - 1)) + j;
    const int other = __shfl(id, from);
    const float od = __shfl(d, from);
    all += other == id ? od : 0.0f;
  }
  V* const to = grad + (int64_t)t * ld + id;
  if (accumulate) {
    if (on) all += (float)*to;
  } else {
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // the zeros come first
  }
  if (on) *to = (V)all;
}

}  // namespace

hipError_t launch_route_backward(const int32_t* idx, const float* w, const float* grad_w, int T,
                                 int E, int K, bool accumulate, void* grad_logits, int dtype,
                                 int64_t ld, hipStream_t s) {
  auto go = [&](auto kernel, int tokens) {
    const dim3 grid((T + kWaves * tokens - 1) / (kWaves * tokens));
    kernel<<<grid, kWaves * 64, 0, s>>>(idx, w, grad_w, T, E, K, accumulate, grad_logits, ld);
  };
  auto type = [&](auto DT) {
    constexpr int dt = decltype(DT)::value;
    if (K <= 16)
      go(route_backward_kernel<dt, 16>, 4);
    else if (K <= 32)
      go(route_backward_kernel<dt, 32>, 2);
    else
      go(route_backward_kernel<dt, 64>, 1);
  };
  if (dtype == kF32)
    type(std::integral_constant<int, kF32>());
  else if (dtype == kBF16)
    type(std::integral_constant<int, kBF16>());
  else
    type(std::integral_constant<int, kF16>());
  return hipGetLastError();
}

}  // namespace moe
