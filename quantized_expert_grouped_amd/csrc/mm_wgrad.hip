// The gradients of the grouped product's weights and bias,
//   dw[e, n, k] = sum_r grad[r, n] a[a(r), k],   db[e, n] = sum_r grad[r, n].
#include "mm_launch.hpp"

namespace moe {

namespace {

template <int DT>
hipError_t wgrad_type(const MmProblem& p, hipStream_t s) {
  return p.out_dtype == DT ? launch_tiles<kMmWgrad, DT, DT, false>(p, s)
                           : launch_tiles<kMmWgrad, DT, kF32, false>(p, s);
}

}  // namespace

size_t mm_wgrad_workspace(int, int, int, int) { return 0; }

hipError_t launch_mm_wgrad(const MmProblem& p_, void*, hipStream_t s) {
  MmProblem p = p_;
  set_division(p);
  return p.dtype == kBF16 ? wgrad_type<kBF16>(p, s) : wgrad_type<kF16>(p, s);
}

}  // namespace moe
