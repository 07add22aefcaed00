// Rows to the experts and back, of any of the three types, with their gradients:
//   dispatch          rows[r] = x[src[r] / K]
//   combine           out[t] = residual[t] + sum_{k < K} w[t, k] rows[slot[t, k]]
//   combine backward  grad_rows[slot[t, k]] = w[t, k] grad_out[t],
//                     grad_w[t, k] = sum_i grad_out[t, i] rows[slot[t, k], i]
// (dispatch's gradient is the combine without weights).  k ascends, sums are fp32 fused
// multiply-adds, each result is rounded once; no row is looked at that no route names.
//
// All are bound by memory.  A thread owns 8 neighbouring columns, and a wavefront lies within one
// token, whose slots and weights are scalars.  Rows may start at any element: the wide loads and
// stores need no more than the element's alignment, and only the last H % 8 columns go one by one.
#include <algorithm>

#include "common.hpp"
#include "train.hpp"

namespace moe {

namespace {

constexpr int kVec = 8;

template <int DT>
struct Cols {
  typedef typename Elem<DT>::type T;
  typedef T vec __attribute__((ext_vector_type(kVec), aligned(sizeof(T))));
};
struct Vals {
  float v[kVec];
};

// n of the 8 columns from `at` on are there (uniform but for a row's last thread)
template <int DT>
__device__ __forceinline__ typename Cols<DT>::vec load(const void* p, int64_t at, int n) {
  typedef typename Cols<DT>::T T;
  typedef typename Cols<DT>::vec vec;
  const T* q = static_cast<const T*>(p) + at;
  vec d = {};
  if (n >= kVec) return *reinterpret_cast<const vec*>(q);
#pragma unroll
  for (int i = 0; i < kVec - 1; ++i)
    if (i < n) d[i] = q[i];
  return d;
}
template <int DT>
__device__ __forceinline__ void store(void* p, int64_t at, int n, const Vals& y) {
  typedef typename Cols<DT>::T T;
  typedef typename Cols<DT>::vec vec;
  T* q = static_cast<T*>(p) + at;
  vec d;
#pragma unroll
  for (int i = 0; i < kVec; ++i) d[i] = (T)y.v[i];
  if (n >= kVec) {
    *reinterpret_cast<vec*>(q) = d;
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec - 1; ++i)
    if (i < n) q[i] = d[i];
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// V: the values' bits
template <class V>
__global__ __launch_bounds__(256) void dispatch_kernel(DispatchArgs a) {
  typedef V vec __attribute__((ext_vector_type(kVec), aligned(sizeof(V))));
  const int r = uniform(blockIdx.x * blockDim.y + threadIdx.y);
  if (r >= a.rows) return;
  const int v = a.src[r], t = v / a.K;
  if (v < 0 || t >= a.T) return;
  const V* x = static_cast<const V*>(a.x) + t * a.ldx;
  V* out = static_cast<V*>(a.out) + r * a.ldo;
  for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * kVec; c < a.H;
       c += gridDim.y * blockDim.x * kVec) {
    if (c + kVec <= a.H)
      *reinterpret_cast<vec*>(out + c) = *reinterpret_cast<const vec*>(x + c);
    else
      for (int i = c; i < a.H; ++i) out[i] = x[i];
  }
}

constexpr int kBatch = 8;  // rows whose loads are under way together

template <int DT, int ODT>
__global__ __launch_bounds__(256) void combine_rows_kernel(CombineArgs a) {
  const int t = uniform(blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= a.T) return;
  const int32_t* slot = a.slot + (int64_t)t * a.K;
  const float* w = a.w ? a.w + (int64_t)t * a.K : nullptr;
  for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * kVec; c < a.H;
       c += gridDim.y * blockDim.x * kVec) {
    const int n = a.H - c;
    Vals acc = {};
    if (a.residual) {
      const auto d = load<ODT>(a.residual, t * a.ldres + c, n);
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc.v[i] = (float)d[i];
    }
    for (int k0 = 0; k0 < a.K; k0 += kBatch) {
      typename Cols<DT>::vec d[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (k0 + j < a.K && (uint32_t)slot[k0 + j] < (uint32_t)a.n_rows)  // uniform
          d[j] = load<DT>(a.rows, slot[k0 + j] * a.ldr + c, n);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (k0 + j < a.K && (uint32_t)slot[k0 + j] < (uint32_t)a.n_rows) {
          const float wk = w ? w[k0 + j] : 1.0f;
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc.v[i] = fmaf(wk, (float)d[j][i], acc.v[i]);
        }
    }
    store<ODT>(a.out, t * a.ldo + c, n, acc);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// A workgroup of blockDim.x threads to a token.
template <int DT, int GDT>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineBackwardArgs a) {
  __shared__ float part[4][kBatch];
  const int t = blockIdx.x, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int32_t* slot = a.slot + (int64_t)t * a.K;
  const float* w = a.w ? a.w + (int64_t)t * a.K : nullptr;
  for (int k0 = 0; k0 < a.K; k0 += kBatch) {
    float dot[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) dot[j] = 0.0f;
    for (int c = threadIdx.x * kVec; c < a.H; c += blockDim.x * kVec) {
      const int n = a.H - c;
      const auto g = load<GDT>(a.grad_out, t * a.ldg + c, n);
      typename Cols<DT>::vec d[kBatch];
      if (a.grad_w)
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (k0 + j < a.K && (uint32_t)slot[k0 + j] < (uint32_t)a.n_rows)
            d[j] = load<DT>(a.rows, slot[k0 + j] * a.ldr + c, n);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (k0 + j < a.K && (uint32_t)slot[k0 + j] < (uint32_t)a.n_rows) {
          if (a.grad_w)
#pragma unroll
            for (int i = 0; i < kVec; ++i) dot[j] = fmaf((float)g[i], (float)d[j][i], dot[j]);
          if (a.grad_rows) {
            const float wk = w ? w[k0 + j] : 1.0f;
            Vals y;
#pragma unroll
            for (int i = 0; i < kVec; ++i) y.v[i] = wk * (float)g[i];
            store<DT>(a.grad_rows, slot[k0 + j] * a.ldgr + c, n, y);
          }
        }
    }
    if (!a.grad_w) continue;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      dot[j] = wave_sum(dot[j]);
      if ((threadIdx.x & 63) == 0) part[wave][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kBatch && k0 + threadIdx.x < a.K) {
      float s = part[0][threadIdx.x];
      for (int i = 1; i < waves; ++i) s += part[i][threadIdx.x];
      a.grad_w[(int64_t)t * a.K + k0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// Threads of a row: a multiple of 64, up to 256; as many rows as make 256 threads.
int row_threads(int H) {
  const int n = (H + kVec - 1) / kVec;
  return n <= 64 ? 64 : n <= 128 ? 128 : 256;
}
struct Shape {
  dim3 grid, block;
};
Shape shape_of(int rows, int H) {
  const int x = row_threads(H), y = 256 / x;
  const int chunks = (H + kVec * x - 1) / (kVec * x);
  return {dim3((rows + y - 1) / y, std::min(chunks, 64)), dim3(x, y)};
}

}  // namespace

hipError_t launch_dispatch_rows(const DispatchArgs& a, hipStream_t s) {
  const Shape g = shape_of(a.rows, a.H);
  if (a.dtype == kF32)
    dispatch_kernel<uint32_t><<<g.grid, g.block, 0, s>>>(a);
  else
    dispatch_kernel<uint16_t><<<g.grid, g.block, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t s) {
  const Shape g = shape_of(a.T, a.H);
  if (a.dtype == kF32)
    combine_rows_kernel<kF32, kF32><<<g.grid, g.block, 0, s>>>(a);
  else if (a.dtype == kBF16 && a.out_dtype == kF32)
    combine_rows_kernel<kBF16, kF32><<<g.grid, g.block, 0, s>>>(a);
  else if (a.dtype == kBF16)
    combine_rows_kernel<kBF16, kBF16><<<g.grid, g.block, 0, s>>>(a);
  else if (a.out_dtype == kF32)
    combine_rows_kernel<kF16, kF32><<<g.grid, g.block, 0, s>>>(a);
  else
    combine_rows_kernel<kF16, kF16><<<g.grid, g.block, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_combine_rows_backward(const CombineBackwardArgs& a, hipStream_t s) {
  const int threads = row_threads(a.H);
  if (a.dtype == kF32)
    combine_backward_kernel<kF32, kF32><<<a.T, threads, 0, s>>>(a);
  else if (a.dtype == kBF16 && a.grad_dtype == kF32)
    combine_backward_kernel<kBF16, kF32><<<a.T, threads, 0, s>>>(a);
  else if (a.dtype == kBF16)
    combine_backward_kernel<kBF16, kBF16><<<a.T, threads, 0, s>>>(a);
  else if (a.grad_dtype == kF32)
    combine_backward_kernel<kF16, kF32><<<a.T, threads, 0, s>>>(a);
  else
    combine_backward_kernel<kF16, kF16><<<a.T, threads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
