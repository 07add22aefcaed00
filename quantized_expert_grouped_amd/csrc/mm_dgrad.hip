// The gradient of the rows that the grouped product read,
//   da[r, k] = sum_n grad[r, n] w[e, n, k],
// or, through the SwiGLU that made them, of its gate and up.
#include "mm_launch.hpp"

namespace moe {

template <int DT>
static hipError_t dgrad(const MmProblem& p, hipStream_t s) {
  return p.swiglu            ? launch_tiles<kMmDgrad, DT, DT, true>(p, s)
         : p.out_dtype == DT ? launch_tiles<kMmDgrad, DT, DT, false>(p, s)
                             : launch_tiles<kMmDgrad, DT, kF32, false>(p, s);
}

hipError_t launch_mm_dgrad(const MmProblem& p, hipStream_t s) {
  return p.dtype == kBF16 ? dgrad<kBF16>(p, s) : dgrad<kF16>(p, s);
}

}  // namespace moe
