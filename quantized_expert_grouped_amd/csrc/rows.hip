// Rows to the experts and back, of any of the three types, with their gradients:
//   dispatch          rows[r] = x[src[r] / K]
//   combine           out[t] = residual[t] + sum_{k < K} w[t, k] rows[slot[t, k]]
//   combine backward  grad_rows[slot[t, k]] = w[t, k] grad_out[t],
//                     grad_w[t, k] = sum_i grad_out[t, i] rows[slot[t, k], i]
// (dispatch's gradient is the combine without weights).  k ascends, sums are fp32 fused
// multiply-adds, each result is rounded once; no row is looked at that no route names.
//
// All are bound by memory.  A thread owns 8 neighbouring columns, and a wavefront lies within one
// row, whose src, or slots and weights, are scalars.  Rows may start at any element: the wide loads
// and stores need no more than the element's alignment, and only the last H % 8 columns go one by
// one.  Rows of the experts are read and written once, so past the caches.
#include <algorithm>

#include "common.hpp"
#include "train.hpp"

namespace moe {

namespace {

constexpr int kVec = 8;

template <class T>
using Vec = T __attribute__((ext_vector_type(kVec), aligned(sizeof(T))));

// 8 columns from p on, of which n are there (all, but for a row's last thread).
template <class T>
__device__ __forceinline__ Vec<T> load(const T* p, int n) {
  if (n >= kVec) return __builtin_nontemporal_load(reinterpret_cast<const Vec<T>*>(p));
  Vec<T> d = {};
#pragma unroll
  for (int i = 0; i < kVec - 1; ++i)
    if (i < n) d[i] = p[i];
  return d;
}
template <class T>
__device__ __forceinline__ void store(T* p, int n, const Vec<T>& d) {
  if (n >= kVec) {
    __builtin_nontemporal_store(d, reinterpret_cast<Vec<T>*>(p));
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec - 1; ++i)
    if (i < n) p[i] = d[i];
}
template <class T>
__device__ __forceinline__ Vec<T> rounded(const float (&y)[kVec]) {
  Vec<T> d;
#pragma unroll
  for (int i = 0; i < kVec; ++i) d[i] = (T)y[i];
  return d;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// what a wavefront's scalars are read by, whatever is written meanwhile
template <class T>
using Scalars = const __attribute__((address_space(4))) T*;
template <class T>
__device__ __forceinline__ Scalars<T> scalars(const T* p) {
  return (Scalars<T>)(uintptr_t)p;
}

// kRows rows a thread, whose loads are under way together.  Bound by memory: 73,800 rows of 2048 bf16
// of 8192 tokens take 84 us, 604 MB read and written, the reads mostly from the memory-side cache.
// V: the values' bits.
template <class V, int kRows>
__global__ __launch_bounds__(256) void dispatch_kernel(DispatchArgs a) {
  const int r0 = uniform((blockIdx.x * blockDim.y + threadIdx.y) * kRows);
  int t[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int v = scalars(a.src)[min(r0 + j, a.rows - 1)];
    t[j] = r0 + j >= a.rows || v < 0 || v / a.K >= a.T ? -1 : v / a.K;
  }
  const V* x = static_cast<const V*>(a.x);
  V* out = static_cast<V*>(a.out);
  for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * kVec; c < a.H;
       c += gridDim.y * blockDim.x * kVec) {
    const int n = a.H - c;
    Vec<V> d[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const V* from = x + max(t[j], 0) * a.ldx + c;  // read K times: through the caches
      d[j] = n >= kVec ? *reinterpret_cast<const Vec<V>*>(from) : load(from, n);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (t[j] >= 0) store(out + (r0 + j) * a.ldo + c, n, d[j]);
  }
}

// Routes whose rows' loads are under way together.
template <int DT>
constexpr int kBatch = DT == kF32 ? 8 : 16;

template <int DT, int ODT>
__global__ __launch_bounds__(256) void combine_rows_kernel(CombineArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<ODT>::type OT;
  constexpr int kB = kBatch<DT>;
  const int t = uniform(blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= a.T) return;
  const auto slot = scalars(a.slot) + (int64_t)t * a.K;
  const auto w = scalars(a.w) + (a.w ? (int64_t)t * a.K : 0);
  const T* rows = static_cast<const T*>(a.rows);
  for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * kVec; c < a.H;
       c += gridDim.y * blockDim.x * kVec) {
    const int n = a.H - c;
    float acc[kVec] = {};
    if (a.residual) {
      const Vec<OT> d = load(static_cast<const OT*>(a.residual) + t * a.ldres + c, n);
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = (float)d[i];
    }
    for (int k0 = 0; k0 < a.K; k0 += kB) {
      Vec<T> d[kB];
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (k0 + j < a.K && (uint32_t)slot[k0 + j] < (uint32_t)a.n_rows)  // uniform
          d[j] = load(rows + slot[k0 + j] * a.ldr + c, n);
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (k0 + j < a.K && (uint32_t)slot[k0 + j] < (uint32_t)a.n_rows) {
          const float wk = a.w ? w[k0 + j] : 1.0f;
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] = fmaf(wk, (float)d[j][i], acc[i]);
        }
    }
    store(static_cast<OT*>(a.out) + t * a.ldo + c, n, rounded<OT>(acc));
  }
}

// The wavefront's sum, in all lanes: DPP steps leave each row of 16 lanes with its row's, then the
// four rows' are read into scalars.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v += dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v += dpp<0x141>(v);  // lane i <-> 7 - i within each half row
  v += dpp<0x140>(v);  // lane i <-> 15 - i within each row
  auto row = [&](int i) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * i));
  };
  return (row(0) + row(1)) + (row(2) + row(3));
}

// A workgroup of blockDim.x threads to a token (a wavefront to a token: 199 us instead of 148 at 8192
// tokens, K = 10, H = 2048, bf16 rows, fp32 gradients).  Bound by memory: 738 MB, 5.0 TB/s.
template <int DT, int GDT>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineBackwardArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<GDT>::type GT;
  constexpr int kB = kBatch<DT>;
  __shared__ float part[4][kB];
  const int wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6, t = blockIdx.x;
  const auto slot = scalars(a.slot) + (int64_t)t * a.K;
  const auto w = scalars(a.w) + (a.w ? (int64_t)t * a.K : 0);
  const T* rows = static_cast<const T*>(a.rows);
  T* grad_rows = static_cast<T*>(a.grad_rows);
  for (int k0 = 0; k0 < a.K; k0 += kB) {
    float dot[kB];
#pragma unroll
    for (int j = 0; j < kB; ++j) dot[j] = 0.0f;
    for (int c = threadIdx.x * kVec; c < a.H; c += blockDim.x * kVec) {
      const int n = a.H - c;
      Vec<T> d[kB];
      if (a.grad_w)
#pragma unroll
        for (int j = 0; j < kB; ++j)
          if (k0 + j < a.K && (uint32_t)slot[k0 + j] < (uint32_t)a.n_rows)
            d[j] = load(rows + slot[k0 + j] * a.ldr + c, n);
      const Vec<GT> gv = load(static_cast<const GT*>(a.grad_out) + t * a.ldg + c, n);
      float g[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) g[i] = (float)gv[i];
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (k0 + j < a.K && (uint32_t)slot[k0 + j] < (uint32_t)a.n_rows) {
          if (a.grad_w)
#pragma unroll
            for (int i = 0; i < kVec; ++i) dot[j] = fmaf(g[i], (float)d[j][i], dot[j]);
          if (grad_rows) {
            const float wk = a.w ? w[k0 + j] : 1.0f;
            float y[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) y[i] = wk * g[i];
            store(grad_rows + slot[k0 + j] * a.ldgr + c, n, rounded<T>(y));
          }
        }
    }
    if (!a.grad_w) continue;
    float* to = a.grad_w + (int64_t)t * a.K + k0;
    const int many = min(kB, a.K - k0);
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      if (j < many) {  // uniform
        const float s = wave_sum(dot[j]);
        if ((threadIdx.x & 63) == 0) part[wave][j] = s;
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < many) {
      float s = part[0][threadIdx.x];
      for (int i = 1; i < waves; ++i) s += part[i][threadIdx.x];
      to[threadIdx.x] = s;
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
Shape shape_of(int rows, int H, int rows_a_thread) {
  const int x = row_threads(H), y = 256 / x, high = y * rows_a_thread;
  const int chunks = (H + kVec * x - 1) / (kVec * x);
  return {dim3((rows + high - 1) / high, std::min(chunks, 64)), dim3(x, y)};
}

template <class V>
void dispatch(const DispatchArgs& a, hipStream_t s) {
  // Few rows: one a thread, for more workgroups (kernels in a row, one and four rows a thread, us: 170
  // rows of 2048 bf16 2.0, 2.7; 2000 rows 3.5, 3.7; 4000 rows 4.6, 4.6; 8000 rows 7.1, 6.7; of 8192
  // values 600 rows 3.7, 4.0, 2000 rows 7.3, 7.0, 8000 rows 30.8, 31.4; 80,000 rows of 256 14.9, 11.6,
  // of 2048 86.5, 89.5).
  if (a.rows < 4096) {
    const Shape g = shape_of(a.rows, a.H, 1);
    dispatch_kernel<V, 1><<<g.grid, g.block, 0, s>>>(a);
  } else {
    const Shape g = shape_of(a.rows, a.H, 4);
    dispatch_kernel<V, 4><<<g.grid, g.block, 0, s>>>(a);
  }
}

template <int DT, int GDT>
void backward(const CombineBackwardArgs& a, hipStream_t s) {
  combine_backward_kernel<DT, GDT><<<a.T, row_threads(a.H), 0, s>>>(a);
}

}  // namespace

hipError_t launch_dispatch_rows(const DispatchArgs& a, hipStream_t s) {
  if (a.dtype == kF32)
    dispatch<uint32_t>(a, s);
  else
    dispatch<uint16_t>(a, s);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t s) {
  const Shape g = shape_of(a.T, a.H, 1);
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
  if (a.dtype == kF32)
    backward<kF32, kF32>(a, s);
  else if (a.dtype == kBF16 && a.grad_dtype == kF32)
    backward<kBF16, kF32>(a, s);
  else if (a.dtype == kBF16)
    backward<kBF16, kBF16>(a, s);
  else if (a.grad_dtype == kF32)
    backward<kF16, kF32>(a, s);
  else
    backward<kF16, kF16>(a, s);
  return hipGetLastError();
}

}  // namespace moe
