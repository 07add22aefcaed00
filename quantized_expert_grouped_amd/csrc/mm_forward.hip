// The grouped product of 16-bit rows and weights,
//   y[r, n] = sum_k a[a(r), k] w[e, n, k] + bias[e, n]
// with a residual, or with the SwiGLU of gate and up, in its epilogue.
#include "mm_launch.hpp"
#include "mm_narrow.hpp"

namespace moe {

template <int DT, int ODT, bool SWIGLU>
static hipError_t forward_any(const MmProblem& p, hipStream_t s) {
  return narrow::wins(p) ? narrow::launch<DT, ODT, SWIGLU>(p, s)
                         : launch_tiles<kMmForward, DT, ODT, SWIGLU>(p, s);
}
template <int DT>
static hipError_t forward(const MmProblem& p, hipStream_t s) {
  return p.swiglu            ? forward_any<DT, DT, true>(p, s)
         : p.out_dtype == DT ? forward_any<DT, DT, false>(p, s)
                             : forward_any<DT, kF32, false>(p, s);
}

hipError_t launch_mm_forward(const MmProblem& p_, hipStream_t s) {
  MmProblem p = p_;
  p.by_k = division_by(p.K);
  return p.dtype == kBF16 ? forward<kBF16>(p, s) : forward<kF16>(p, s);
}

}  // namespace moe
