// The activation row that a route reads: route / K by a product and a shift, in bounds whatever the
// route is.  Plain C++ (constexpr functions are device functions, too), so a host test covers it.
#pragma once

#include <stdint.h>

namespace moe {

// n / K = n * mul >> shift for 0 <= n < 2^31 and K = 1 .. 64: with 2^(s - 1) < K <= 2^s, shift = 31 + s
// and mul = 2^shift / K + 1 < 2^32, mul K exceeds 2^shift by at most K <= 2^s, so n * mul / 2^shift
// exceeds n / K by less than 1 / K.
struct Division {
  uint32_t mul, shift;
};
constexpr Division division_by(int K) {
  uint32_t shift = 31;
  while (1 << (shift - 31) < K) ++shift;
  return {(uint32_t)(((uint64_t)1 << shift) / (uint32_t)K + 1), shift};
}

// The nearest one of n_act rows for a route outside [0, n_act K).
constexpr int route_row(int32_t route, uint32_t mul, uint32_t shift, int n_act) {
  const int row = route < 0 ? 0 : (int)((uint64_t)(uint32_t)route * mul >> shift);
  return row < n_act ? row : n_act - 1;
}

}  // namespace moe
