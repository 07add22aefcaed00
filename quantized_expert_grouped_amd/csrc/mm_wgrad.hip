// The gradients of the grouped product's weights and bias,
//   dw[e, n, k] = sum_r grad[r, n] a[a(r), k],   db[e, n] = sum_r grad[r, n].
// Where the matrices have too few tiles for the CUs, each expert's rows are taken in parts, whose fp32
// sums lie in the workspace and are joined, in order, by a second launch.
#include "mm_launch.hpp"

namespace moe {

namespace {

// Which tile, and how many parts of an expert's rows, by sizes alone.  A part has 256 rows at least
// in the mean.  8192 rows of one expert, us with one part and as chosen: 64 x 64 89, 13; 512 x 512
// 102, 25; 1024 x 1024 104, 35; 2048 x 2048 129, 91; four experts of 512 x 512 55, 26.
struct Plan {
  bool large;
  int parts;
};
template <class G>
int64_t tiles_of(int n_out, int k_in, int E) {
  return (int64_t)((n_out + G::BJ - 1) / G::BJ) * ((k_in + G::BI - 1) / G::BI) * E;
}
Plan plan(int rows, int n_out, int k_in, int E) {
  const int64_t large = tiles_of<Large<kMmWgrad>>(n_out, k_in, E);
  const int64_t small = tiles_of<Small<kMmWgrad>>(n_out, k_in, E);
  Plan p{large >= kCus / 4, 1};
  const int64_t fit = p.large ? kCus / large : 2 * kCus / small;
  p.parts = (int)std::max<int64_t>(1, std::min<int64_t>(fit, rows / ((int64_t)E * 256)));
  if (p.large && p.parts == 1 && large < kCus) p.large = false;  // few rows, too
  return p;
}

// out[e, x] = the sum of its parts' [e, s, x], x in fours; w and then b.
template <int ODT>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ w,
                                                   const float* __restrict__ b, int parts,
                                                   int64_t nw, int64_t nb, int64_t all, void* out,
                                                   void* out_b) {
  int64_t x = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (x >= all) return;
  const int64_t all_w = all / (nw + nb) * nw;
  const bool bias = x >= all_w;
  if (bias) x -= all_w;
  const int64_t n = bias ? nb : nw, e = x / n;
  const float* from = (bias ? b : w) + (e * parts) * n + (x - e * n);
  v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int kBatch = 8;
  for (int s0 = 0; s0 < parts; s0 += kBatch) {
    v4f v[kBatch];
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (s0 + s < parts) v[s] = *reinterpret_cast<const v4f*>(from + (s0 + s) * n);
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (s0 + s < parts) y += v[s];
  }
  store4<ODT>(bias ? out_b : out, x, y);
}

template <int DT, int ODT>
hipError_t run(const MmProblem& p, bool large, hipStream_t s) {
  return large ? launch_geo<kMmWgrad, DT, ODT, false, Large<kMmWgrad>>(p, s)
               : launch_small<kMmWgrad, DT, ODT, false>(p, s);
}
template <int DT>
hipError_t wgrad(MmProblem p, void* ws, hipStream_t s) {
  const Plan plan_ = plan(p.rows, p.n_out, p.k_in, p.E);
  p.parts = plan_.parts;
  if (p.parts == 1)
    return p.out_dtype == DT ? run<DT, DT>(p, plan_.large, s) : run<DT, kF32>(p, plan_.large, s);
  void *out = p.out, *out_b = p.bias_out;
  const int64_t nw = (int64_t)p.n_out * p.k_in, nb = p.bias_out ? p.n_out : 0;
  float* const w = static_cast<float*>(ws);
  float* const b = w + p.E * p.parts * nw;
  p.out = w;
  if (out_b) p.bias_out = b;
  const hipError_t e = run<DT, kF32>(p, plan_.large, s);
  if (e != hipSuccess) return e;
  const int64_t all = p.E * (nw + nb);
  const unsigned grid = (unsigned)((all / 4 + 255) / 256);
  if (p.out_dtype == DT)
    join_kernel<DT><<<grid, 256, 0, s>>>(w, b, p.parts, nw, nb, all, out, out_b);
  else
    join_kernel<kF32><<<grid, 256, 0, s>>>(w, b, p.parts, nw, nb, all, out, out_b);
  return hipGetLastError();
}

}  // namespace

size_t mm_wgrad_workspace(int rows, int n_out, int k_in, int E) {
  const int parts = plan(rows, n_out, k_in, E).parts;
  return parts == 1 ? 0 : (size_t)E * parts * ((size_t)n_out * k_in + n_out) * sizeof(float);
}

hipError_t launch_mm_wgrad(const MmProblem& p_, void* ws, hipStream_t s) {
  MmProblem p = p_;
  p.by_k = division_by(p.K);
  return p.dtype == kBF16 ? wgrad<kBF16>(p, ws, s) : wgrad<kF16>(p, ws, s);
}

}  // namespace moe
