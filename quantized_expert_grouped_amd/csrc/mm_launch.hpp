// The tile kernel's launch, for the sources that instantiate it, one to an operation.
#pragma once

#include <algorithm>

#include "mm_tile.hpp"

namespace moe {

template <int OP, int DT, int ODT, bool SWIGLU, class G>
__global__ __launch_bounds__(G::kWaves * 64, 2) void mm_kernel(MmProblem p) {
  typedef tile::Kernel<OP, DT, ODT, SWIGLU, G> K;
  __shared__ typename K::L lds;
  K(p, lds).run();
}

constexpr int kCus = 256;  // MI355X

// A bound of the tiles there are, whatever the offsets.
template <class G>
int64_t most_tiles(const MmProblem& p) {
  const int feat = p.op == kMmForward && p.swiglu ? G::BI / 2 : G::BI;
  const int64_t ni = ((p.op == kMmForward ? p.n_out : p.k_in) + feat - 1) / feat;
  if (p.op == kMmWgrad) return ni * ((p.n_out + G::BJ - 1) / G::BJ) * p.E;
  return ni * (p.rows / G::BJ + std::min(p.E, p.rows));
}

template <int OP, int DT, int ODT, bool SWIGLU, class G>
hipError_t launch_geo(const MmProblem& p, hipStream_t s) {
  const int64_t most = (most_tiles<G>(p) + 7) / 8 * 8;
  const unsigned grid = (unsigned)std::min<int64_t>(most, kCus * G::kPerCu);
  mm_kernel<OP, DT, ODT, SWIGLU, G><<<grid, G::kWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}
typedef tile::Geo<4, 2, 2, 4> Large;  // 256 x 256
typedef tile::Geo<2, 2, 2, 2> Small;  // 128 x 128, two workgroups a CU

template <int OP, int DT, int ODT, bool SWIGLU>
hipError_t launch_tiles(const MmProblem& p, hipStream_t s) {
  return most_tiles<Large>(p) >= kCus ? launch_geo<OP, DT, ODT, SWIGLU, Large>(p, s)
                                      : launch_geo<OP, DT, ODT, SWIGLU, Small>(p, s);
}

}  // namespace moe
