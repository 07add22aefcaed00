// The router's load-balance loss, its per-expert counts and its gradient.  With p[t] = softmax of
// token t's E logits, n the valid tokens, c[e] how many of their K routes each went to expert e:
//   f[e] = c[e] / (n K),   P[e] = (1/n) sum_t p[t, e],   loss = E sum_e f[e] P[e],
//   d loss / d logits[t, j] = (E / n) p[t, j] (f[j] - sum_e f[e] p[t, e]),
// the counts being constants of the gradient.  Since sum_e p[t, e] = 1, f may be replaced by
// f - 1/E in the bracket, and is: near balance f is almost constant and the bracket a small
// difference of large terms otherwise.  f[e] - 1/E = (c[e] E - N) / (E n K), N = sum c, exact integers
// up to one rounding.
//
// A row of logits is one wavefront's, read once into registers (-inf: an expert that the token may not
// take; a row of nothing else has p = 0).  Forward: each workgroup keeps its rows' sums of p per
// column in registers and its counts in LDS and leaves one row of partial sums; a second launch adds
// those in a fixed order, so results do not change from run to run, and its last workgroup (an integer ticket)
// forms the loss.
#include <math.h>

#include "common.hpp"
#include "mx.hpp"

namespace moe {

namespace {

constexpr int kWaves = 16;  // wavefronts of a forward workgroup

// Workspace: ticket, then per workgroup valid tokens, counts [E], sums [E].
struct Partials {
  int32_t* ticket;
  int32_t* tokens;  // [groups]
  int32_t* counts;  // [groups x E]
  float* sums;      // [groups x E]
};
__host__ __device__ inline Partials partials(void* ws, int groups, int E) {
  Partials q;
  q.ticket = static_cast<int32_t*>(ws);
  q.tokens = q.ticket + 64;
  q.counts = q.tokens + kBalanceGroups;
  q.sums = reinterpret_cast<float*>(q.counts + (size_t)groups * E);
  return q;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Lane l's columns of a row are j * 64 + l, j < VPL.  Gives exp(x - max) and 1 / their sum, 0 for a row
// with nothing above -inf.
template <int DT, int VPL>
__device__ __forceinline__ float row_softmax(const void* logits, int64_t at, int E, float (&p)[VPL]) {
  typedef typename Elem<DT>::type T;
  const int lane = threadIdx.x & 63;
  const T* l = static_cast<const T*>(logits) + at;
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = j * 64 + lane;
    p[j] = c < E ? (float)l[c] : -INFINITY;
    m = fmaxf(m, p[j]);
  }
  m = wave_max(m);
  if (m == -INFINITY) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) p[j] = 0.0f;
    return 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    p[j] = expf(p[j] - m);
    s += p[j];
  }
  return 1.0f / wave_sum(s);
}

template <int DT, int VPL>
__global__ __launch_bounds__(kWaves * 64) void balance_rows_kernel(BalanceArgs a, void* ws) {
  __shared__ int32_t hist[VPL * 64];
  __shared__ float sums[VPL * 64];
  __shared__ int32_t tokens;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Partials q = partials(ws, gridDim.x, a.E);
  for (int e = threadIdx.x; e < VPL * 64; e += kWaves * 64) {
    hist[e] = 0;
    sums[e] = 0.0f;
  }
  if (threadIdx.x == 0) {
    tokens = 0;
    if (blockIdx.x == 0) *q.ticket = 0;
  }
  __syncthreads();
  float acc[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) acc[j] = 0.0f;
  int mine = 0;
  for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.T; t += (int64_t)gridDim.x * kWaves) {
    if (a.valid && a.valid[t] == 0) continue;  // uniform
    ++mine;
    if (lane < a.K) {
      const int e = a.idx[t * a.K + lane];
      if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
    }
    float p[VPL];
    const float r = row_softmax<DT, VPL>(a.logits, t * a.ld, a.E, p);
#pragma unroll
    for (int j = 0; j < VPL; ++j) acc[j] = fmaf(p[j], r, acc[j]);
  }
  if (lane == 0 && mine) atomicAdd(&tokens, mine);
  for (int wv = 0; wv < kWaves; ++wv) {  // in the wavefronts' order
    if (wave == wv)
#pragma unroll
      for (int j = 0; j < VPL; ++j) sums[j * 64 + lane] += acc[j];
    __syncthreads();
  }
  for (int e = threadIdx.x; e < a.E; e += kWaves * 64) {
    q.counts[(size_t)blockIdx.x * a.E + e] = hist[e];
    q.sums[(size_t)blockIdx.x * a.E + e] = sums[e];
  }
  if (threadIdx.x == 0) q.tokens[blockIdx.x] = tokens;
}

// 32 columns by 8 strands of workgroups' partial rows.
__global__ __launch_bounds__(256) void balance_join_kernel(int E, int K, int groups, void* ws,
                                                           int32_t* __restrict__ counts,
                                                           float* __restrict__ prob_mean,
                                                           float* __restrict__ loss) {
  __shared__ int32_t c8[8][32];
  __shared__ float s8[8][32];
  __shared__ int32_t n4[4];
  __shared__ bool last;
  const Partials q = partials(ws, groups, E);
  const int col = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + col;
  int n = threadIdx.x < groups ? q.tokens[threadIdx.x] : 0;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o);
  if ((threadIdx.x & 63) == 0) n4[threadIdx.x >> 6] = n;
  int32_t c = 0;
  float s = 0.0f;
  if (e < E)
    for (int g = strand; g < groups; g += 8) {
      c += q.counts[(size_t)g * E + e];
      s += q.sums[(size_t)g * E + e];
    }
  c8[strand][col] = c;
  s8[strand][col] = s;
  __syncthreads();
  n = n4[0] + n4[1] + n4[2] + n4[3];
  if (strand == 0 && e < E) {
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      c += c8[i][col];
      s += s8[i][col];
    }
    counts[e] = c;
    prob_mean[e] = n > 0 ? s / (float)n : 0.0f;
  }
  if (threadIdx.x == 0 && blockIdx.x == 0) counts[E] = n;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(q.ticket, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // loss = E sum_e f[e] P[e]: 256 strands of columns, then a tree, a fixed order
  float v = 0.0f;
  for (int i = threadIdx.x; i < E; i += 256) {
    const int32_t ci = __hip_atomic_load(counts + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const float pi = __hip_atomic_load(prob_mean + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    v = fmaf((float)ci, pi, v);
  }
  v = wave_sum(v);
  __shared__ float v4[4];
  if ((threadIdx.x & 63) == 0) v4[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    *loss = n > 0 ? ((v4[0] + v4[1]) + (v4[2] + v4[3])) * ((float)E / ((float)n * (float)K)) : 0.0f;
}

template <int DT, int VPL>
__global__ __launch_bounds__(256) void balance_backward_kernel(BalanceArgs a,
                                                               const int32_t* __restrict__ counts,
                                                               const float* __restrict__ grad_loss,
                                                               void* __restrict__ grad,
                                                               int64_t ld_grad) {
  typedef typename Elem<DT>::type T;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = counts[a.E];
  float dev[VPL];
  int64_t total = 0;
  int32_t c[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 64 + lane;
    c[j] = e < a.E ? counts[e] : 0;
    total += c[j];
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o);
  // (E / n) (f - 1/E) = (c E - N) / (n n K)
  const float nf = (float)n;
  const float scale = n > 0 ? (grad_loss ? *grad_loss : 1.0f) / (nf * (float)a.K) / nf : 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) dev[j] = (float)((int64_t)c[j] * a.E - total) * scale;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.T; t += (int64_t)gridDim.x * 4) {
    T* g = static_cast<T*>(grad) + t * ld_grad;
    float p[VPL];
    float r = 0.0f, dot = 0.0f;
    const bool on = !a.valid || a.valid[t] != 0;  // uniform
    if (on) {
      r = row_softmax<DT, VPL>(a.logits, t * a.ld, a.E, p);
#pragma unroll
      for (int j = 0; j < VPL; ++j) dot = fmaf(p[j], dev[j], dot);
      dot = wave_sum(dot) * r;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = j * 64 + lane;
      if (e < a.E) g[e] = on ? (T)(p[j] * r * (dev[j] - dot)) : (T)0.0f;
    }
  }
}

template <int DT>
hipError_t forward(const BalanceArgs& a, int groups, void* ws, hipStream_t s) {
  const int vpl = (a.E + 63) / 64;
  if (vpl <= 1) balance_rows_kernel<DT, 1><<<groups, kWaves * 64, 0, s>>>(a, ws);
  else if (vpl <= 2) balance_rows_kernel<DT, 2><<<groups, kWaves * 64, 0, s>>>(a, ws);
  else if (vpl <= 4) balance_rows_kernel<DT, 4><<<groups, kWaves * 64, 0, s>>>(a, ws);
  else if (vpl <= 8) balance_rows_kernel<DT, 8><<<groups, kWaves * 64, 0, s>>>(a, ws);
  else if (vpl <= 16) balance_rows_kernel<DT, 16><<<groups, kWaves * 64, 0, s>>>(a, ws);
  else balance_rows_kernel<DT, 32><<<groups, kWaves * 64, 0, s>>>(a, ws);
  return hipGetLastError();
}

template <int DT>
hipError_t backward(const BalanceArgs& a, const int32_t* counts, const float* grad_loss, void* grad,
                    int64_t ld, hipStream_t s) {
  const int vpl = (a.E + 63) / 64;
  const int grid = a.T / 4 + 1 < 2048 ? a.T / 4 + 1 : 2048;
  if (vpl <= 1) balance_backward_kernel<DT, 1><<<grid, 256, 0, s>>>(a, counts, grad_loss, grad, ld);
  else if (vpl <= 2) balance_backward_kernel<DT, 2><<<grid, 256, 0, s>>>(a, counts, grad_loss, grad, ld);
  else if (vpl <= 4) balance_backward_kernel<DT, 4><<<grid, 256, 0, s>>>(a, counts, grad_loss, grad, ld);
  else if (vpl <= 8) balance_backward_kernel<DT, 8><<<grid, 256, 0, s>>>(a, counts, grad_loss, grad, ld);
  else if (vpl <= 16) balance_backward_kernel<DT, 16><<<grid, 256, 0, s>>>(a, counts, grad_loss, grad, ld);
  else balance_backward_kernel<DT, 32><<<grid, 256, 0, s>>>(a, counts, grad_loss, grad, ld);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_balance_loss(const BalanceArgs& a, int32_t* counts, float* prob_mean, float* loss,
                               void* ws, hipStream_t s) {
  const int groups = balance_groups(a.T);
  hipError_t e = a.dtype == kF32    ? forward<kF32>(a, groups, ws, s)
                 : a.dtype == kBF16 ? forward<kBF16>(a, groups, ws, s)
                                    : forward<kF16>(a, groups, ws, s);
  if (e != hipSuccess) return e;
  balance_join_kernel<<<(a.E + 31) / 32, 256, 0, s>>>(a.E, a.K, groups, ws, counts, prob_mean, loss);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, const int32_t* counts,
                                   const float* grad_loss, void* grad, int64_t ld_grad,
                                   hipStream_t s) {
  return a.dtype == kF32    ? backward<kF32>(a, counts, grad_loss, grad, ld_grad, s)
         : a.dtype == kBF16 ? backward<kBF16>(a, counts, grad_loss, grad, ld_grad, s)
                            : backward<kF16>(a, counts, grad_loss, grad, ld_grad, s);
}

}  // namespace moe
