// The gradient of the router's logits.  The K routing weights are the softmax of the K chosen
// logits, so with gw = d loss / d w
//   d loss / d logits[t, idx[t, k]] = w_k (gw_k - sum_j w_j gw_j),
// and 0 for the other experts.  A route whose id is outside [0, E) has no expert row: its gw counts
// as 0.
//
// A wavefront to a token: lane k holds route k, and the row is built in LDS, then written in whole
// lines.  Bound by those writes.
#include "common.hpp"
#include "train.hpp"

namespace moe {

namespace {

constexpr int kWaves = 4;

template <int DT>
__global__ __launch_bounds__(kWaves * 64) void route_backward_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ w, const float* __restrict__ grad_w,
    int T, int E, int K, bool accumulate, void* grad_logits, int64_t ld) {
  typedef typename Elem<DT>::type V;
  extern __shared__ float row_lds[];  // [kWaves][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * kWaves + wave;
  if (t >= T) return;
  float* row = row_lds + wave * E;
  int id = -1;
  float wk = 0.0f, gw = 0.0f;
  if (lane < K) {
    id = idx[(int64_t)t * K + lane];
    wk = w[(int64_t)t * K + lane];
    if (id >= 0 && id < E) gw = grad_w[(int64_t)t * K + lane];
  }
  float sum = wk * gw;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  const float d = wk * (gw - sum);
  // the wavefront's own LDS row, whose operations complete in order
  for (int e = lane; e < E; e += 64) row[e] = 0.0f;
  __builtin_amdgcn_wave_barrier();
  for (int k = 0; k < K; ++k) {  // one by one: an id may come twice
    if (lane == k && id >= 0 && id < E) row[id] += d;
    __builtin_amdgcn_wave_barrier();
  }
  V* out = static_cast<V*>(grad_logits) + t * ld;
  for (int e = lane; e < E; e += 64)
    out[e] = (V)(accumulate ? (float)out[e] + row[e] : row[e]);
}

}  // namespace

hipError_t launch_route_backward(const int32_t* idx, const float* w, const float* grad_w, int T,
                                 int E, int K, bool accumulate, void* grad_logits, int dtype,
                                 int64_t ld, hipStream_t s) {
  const dim3 grid((T + kWaves - 1) / kWaves);
  const size_t lds = (size_t)kWaves * E * sizeof(float);
  auto go = [&](auto kernel) {
    kernel<<<grid, kWaves * 64, lds, s>>>(idx, w, grad_w, T, E, K, accumulate, grad_logits, ld);
  };
  if (dtype == kF32)
    go(route_backward_kernel<kF32>);
  else if (dtype == kBF16)
    go(route_backward_kernel<kBF16>);
  else
    go(route_backward_kernel<kF16>);
  return hipGetLastError();
}

}  // namespace moe
