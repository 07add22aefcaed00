// The gradients of the grouped product's weights and bias,
//   dw[e, n, k] = sum_r grad[r, n] a[a(r), k],   db[e, n] = sum_r grad[r, n].
#include "mm_launch.hpp"

namespace moe {

namespace {

// Bias gradient: a thread sums 4 columns of an expert's rows.
template <int DT, int ODT>
__global__ __launch_bounds__(64) void mm_bias_kernel(MmProblem p) {
  const int e = blockIdx.x, n = (blockIdx.y * 64 + threadIdx.x) * 4;
  if (n >= p.n_out) return;
  const int last = min(p.offsets[e + 1], p.rows);
  v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int r = p.offsets[e]; r < last; ++r) y += load4<DT>(p.grad, r * p.ldg + n);
  store4<ODT>(p.bias_out, (int64_t)e * p.n_out + n, y);
}

template <int DT, int ODT>
hipError_t wgrad(const MmProblem& p, hipStream_t s) {
  hipError_t e = launch_tiles<kMmWgrad, DT, ODT, false>(p, s);
  if (e == hipSuccess && p.bias_out) {
    mm_bias_kernel<DT, ODT><<<dim3(p.E, (p.n_out + 255) / 256), 64, 0, s>>>(p);
    e = hipGetLastError();
  }
  return e;
}
template <int DT>
hipError_t wgrad_type(const MmProblem& p, hipStream_t s) {
  return p.out_dtype == DT ? wgrad<DT, DT>(p, s) : wgrad<DT, kF32>(p, s);
}

}  // namespace

size_t mm_wgrad_workspace(int, int, int, int) { return 0; }

hipError_t launch_mm_wgrad(const MmProblem& p_, void*, hipStream_t s) {
  MmProblem p = p_;
  set_division(p);
  return p.dtype == kBF16 ? wgrad_type<kBF16>(p, s) : wgrad_type<kF16>(p, s);
}

}  // namespace moe
