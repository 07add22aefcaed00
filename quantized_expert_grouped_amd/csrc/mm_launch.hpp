// The tile kernel's launch, for the sources that instantiate it, one to an operation.
#pragma once

#include <algorithm>

#include "mm_tile.hpp"

namespace moe {

template <int OP, int DT, int ODT, bool SWIGLU, class G>
__global__ __launch_bounds__(G::kWaves * 64, G::kWaves * G::kPerCu / 4) void mm_kernel(MmProblem p) {
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
  if (p.op == kMmWgrad) return ni * ((p.n_out + G::BJ - 1) / G::BJ) * p.E * p.parts;
  return ni * (p.rows / G::BJ + std::min(p.E, p.rows));
}

template <int OP, int DT, int ODT, bool SWIGLU, class G>
hipError_t launch_geo(const MmProblem& p, hipStream_t s) {
  const int64_t most = (most_tiles<G>(p) + 7) / 8 * 8;
  const unsigned grid = (unsigned)std::min<int64_t>(most, kCus * G::kPerCu);
  mm_kernel<OP, DT, ODT, SWIGLU, G><<<grid, G::kWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}
// 256 x 256; 128 x 128 with two workgroups a CU; and, but for wgrad, 128 x 128 with one, where there
// are no more tiles than CUs, and buffers for as many loads on their way as LDS has room for (128 rows,
// 4096 -> 4096: 43 us with two buffers, 38 with four; wgrad of 75 rows in the mean 14.5, 18.9).  In
// stages of 64 a narrow operand's rows come in whole 128-byte lines; wgrad has none, and its short
// tiles like more loads on their way (8191 x 4096 x 4096, and 8192 tokens over 512 experts' 2 x 512 x
// 2048, in us: forward 242 and 585 with stages of 64, 250 and 604 of 32; dgrad 243, 582 and 247, 566;
// wgrad 238, 809 and 239, 779).
template <int OP>
using Large = tile::Geo<4, 2, 2, 4, OP == kMmWgrad ? 32 : 64, OP == kMmWgrad ? 4 : 2>;
template <int OP>
using Small = tile::Geo<2, 2, 2, 2, OP == kMmWgrad ? 32 : 64, OP == kMmWgrad ? 4 : 2>;
template <int OP>
using Deep = tile::Geo<2, 2, 2, 2, 64, 4>;

template <int OP, int DT, int ODT, bool SWIGLU>
hipError_t launch_small(const MmProblem& p, hipStream_t s) {
  if constexpr (OP != kMmWgrad)
    if (most_tiles<Small<OP>>(p) <= kCus) return launch_geo<OP, DT, ODT, SWIGLU, Deep<OP>>(p, s);
  return launch_geo<OP, DT, ODT, SWIGLU, Small<OP>>(p, s);
}
// Large where it fills the CUs and an expert has more than 64 rows in the mean.  In us, 128 x 128 and 256 x
// 256, by rows of each expert (where the border lies goes by the sizes, and none is right for all):
//   512 experts, 2048 -> 2 x 512   forward   40: 374, 413   64: 401, 433   96: 432, 463   160: 607, 520
//                                  dgrad     40: 445, 462   64: 502, 486   96: 519, 503   160: 651, 559
//   64 experts, 2048 -> 2048       forward   40: 132, 139   64: 134, 140   96: 140, 148   160: 184, 159
//                                  dgrad     40: 105, 113   64: 111, 114   96: 121, 122   160: 160, 133
template <int OP, int DT, int ODT, bool SWIGLU>
hipError_t launch_tiles(const MmProblem& p, hipStream_t s) {
  const bool few_rows = p.rows / p.E <= 64;
  return most_tiles<Large<OP>>(p) >= kCus && !few_rows
             ? launch_geo<OP, DT, ODT, SWIGLU, Large<OP>>(p, s)
             : launch_small<OP, DT, ODT, SWIGLU>(p, s);
}

}  // namespace moe
