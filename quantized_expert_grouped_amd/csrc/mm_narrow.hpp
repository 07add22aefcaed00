// The grouped product of few rows: one decoded token's, or a batch's where experts have a few rows
// each.  Bound by the weights' bytes and by latency.
//
// A workgroup takes up to 16 rows of an expert and 16 columns (SwiGLU: 16 gates and their ups); its
// four wavefronts take 128 k's in turn and join their sums in LDS.  Operands go from memory straight
// into v_mfma_f32_16x16x32's layout: lane l holds row l % 16 of an operand, k = 8 (l / 16) .. + 7,
// so a load takes 64 bytes each of 16 rows; the result's lane l has row l % 16 of a and columns
// 4 (l / 16) .. + 3.
#pragma once

#include "mm.hpp"

namespace moe {

namespace narrow {

constexpr int kRows = 16, kCols = 16, kChunk = 128, kWaves = 4;

template <int DT>
__device__ __forceinline__ v4f mfma(const v4i& w, const v4i& a, const v4f& c) {
  typedef typename Half<DT>::v8 v8;
  const v8 x = __builtin_bit_cast(v8, w), y = __builtin_bit_cast(v8, a);
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
}

// The expert of a tile and its rows: tiles of 16 rows are numbered offsets[e] / 16 + e and on, which
// leaves room for all of them, or, with fewer rows than that gives numbers, by their first row.  Some
// numbers belong to no tile.  The lanes compare 64 experts at a time, 512 experts' loads in flight
// together, and what they loaded gives the rows as well: one latency for up to 511 experts.
struct Rows {
  int expert, row0, nrows;
};
__device__ __forceinline__ Rows find(const MmProblem& p, int id, bool by_row) {
  const int lane = threadIdx.x & 63;
  int upto = 0;  // experts whose first number is not above id: a prefix of them
  int first = 0, last = -1;
  for (int e0 = 0; e0 < p.E && last < 0; e0 += 512) {
    int o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = p.offsets[min(e0 + 64 * j + lane, p.E)];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + 64 * j + lane;
      const int n = __popcll(ballot(e < p.E && (by_row ? o[j] : o[j] / kRows + e) <= id));
      if (n > 0) first = __builtin_amdgcn_readlane(o[j], n - 1);
      if (n < 64 && last < 0) last = __builtin_amdgcn_readlane(o[j], n);
      upto += n;
    }
  }
  if (last < 0) last = p.offsets[p.E];  // every expert of a multiple of 64
  Rows t;
  t.expert = max(upto - 1, 0);
  last = min(last, p.rows);
  if (by_row)
    t.row0 = id < first || (id - first) % kRows != 0 ? last : id;
  else
    t.row0 = first + (id - (first / kRows + t.expert)) * kRows;
  t.nrows = min(last - t.row0, kRows);  // <= 0: no tile
  return t;
}

template <int DT, int ODT, bool SWIGLU>
__global__ __launch_bounds__(kWaves * 64) void mm_narrow_kernel(MmProblem p, bool by_row) {
  typedef typename Elem<DT>::type T;
  constexpr int kMats = SWIGLU ? 2 : 1;
  __shared__ v4f part[kWaves - 1][kMats][64];
  const Rows t = find(p, blockIdx.x, by_row);
  if (t.nrows <= 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quarter = lane >> 4, n0 = blockIdx.y * kCols;
  const int64_t row = t.row0 + min(l16, t.nrows - 1);
  const int route = p.src ? p.src[row] : 0;
  const T* w = static_cast<const T*>(p.w) +
               ((int64_t)t.expert * kMats * p.n_out + min(n0 + l16, p.n_out - 1)) * p.k_in +
               8 * quarter;
  const int64_t up = (int64_t)p.n_out * p.k_in;  // from a gate to its up
  const T* a = nullptr;

  v4f acc[kMats];
#pragma unroll
  for (int m = 0; m < kMats; ++m) acc[m] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  // kBatch chunks' loads are under way before the first products, the weights', which need no route,
  // first
  constexpr int kBatch = SWIGLU ? 2 : 4, kStep = kWaves * kChunk;
  for (int c0 = wave * kChunk; c0 < p.k_in; c0 += kBatch * kStep) {
    v4i av[kBatch][4], wv[kBatch][4][kMats];
    // WHOLE: all of the batch is there; otherwise zeros stand for what is past the last k
    auto load = [&](auto WHOLE) {
      auto there = [&](int b, int s) {
        return decltype(WHOLE)::value || c0 + b * kStep + 32 * s + 8 * quarter < p.k_in;
      };
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int m = 0; m < kMats; ++m) {
            wv[b][s][m] = (v4i){0, 0, 0, 0};
            if (there(b, s))
              wv[b][s][m] = __builtin_nontemporal_load(
                  reinterpret_cast<const v4i*>(w + m * up + c0 + b * kStep + 32 * s));
          }
      if (!a)
        a = static_cast<const T*>(p.a) + (p.src ? act_row(p, route) : row) * p.lda + 8 * quarter;
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          av[b][s] = (v4i){0, 0, 0, 0};
          if (there(b, s)) av[b][s] = *reinterpret_cast<const v4i*>(a + c0 + b * kStep + 32 * s);
        }
    };
    if (c0 + (kBatch - 1) * kStep + kChunk <= p.k_in)
      load(std::true_type());
    else
      load(std::false_type());
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int m = 0; m < kMats; ++m) acc[m] = mfma<DT>(wv[b][s][m], av[b][s], acc[m]);
  }
  if (wave > 0)
#pragma unroll
    for (int m = 0; m < kMats; ++m) part[wave - 1][m][lane] = acc[m];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int m = 0; m < kMats; ++m)
    acc[m] = (acc[m] + part[0][m][lane]) + (part[1][m][lane] + part[2][m][lane]);
  const int i = n0 + 4 * quarter;
  if (l16 >= t.nrows || i >= p.n_out) return;
  if (p.bias)
#pragma unroll
    for (int m = 0; m < kMats; ++m)
      acc[m] += load4<DT>(p.bias, ((int64_t)t.expert * kMats + m) * p.n_out + i);
  if constexpr (SWIGLU) {
    const v4f g = acc[0], u = acc[1];
    if (p.z) {
      store4<DT>(p.z, row * p.ldz + i, g);
      store4<DT>(p.z, row * p.ldz + p.n_out + i, u);
    }
    v4f h;
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = g[q] * sigmoid(g[q]) * u[q];
    store4<ODT>(p.out, row * p.ldo + i, h);
  } else {
    v4f y = acc[0];
    if (p.residual) y += load4<ODT>(p.residual, row * p.ldres + i);
    store4<ODT>(p.out, row * p.ldo + i, y);
  }
}

inline int columns(const MmProblem& p) { return (p.n_out + kCols - 1) / kCols; }

// Whether it beats the 128 x 128 tiles, by sizes alone.  It reads a matrix once for each 16 rows, at
// about 4.5 TB/s and 5 us more; a tile of few rows takes 12 us for each 1024 of k, however few there
// are, and reads a matrix once (us, narrow and tiles; rows spread over E experts):
//   4096 -> 4096, E = 1        rows 1: 10, 50   16: 20, 50   64: 46, 53   80: 55, 53   96: 63, 54   128: 80, 40
//   2048 -> 2048, E = 8        2: 7, 27   8: 17, 28   64: 23, 29   96: 25, 29   128: 40, 29
//   1024 -> 1024, E = 64       8: 7, 16   16: 12, 17   24: 14, 18   32: 19, 19   64: 35, 23
//   512 -> 2048, E = 512       10: 8, 10   16: 16, 11   20: 16, 13   80: 54, 31
//   2048 -> 2 x 512, E = 512   10: 14, 18   80: 63, 71   120: 105, 88   160: 121, 119   200: 149, 160   320: 236, 214
// It is taken up to 95, 79, 23, 12 and 170 rows of these.  On the wrong side lie 80 to 95 rows of the first
// (2 us), 80 to 100 of the second (5), 24 of the third (4) and, the times being uneven, 120 (17) and 200 (11)
// of the last.
inline bool wins(const MmProblem& p) {
  if (columns(p) > 65535) return false;
  const int64_t tiles = std::min(p.rows, p.E) + p.rows / kRows;
  const int64_t bytes = tiles * p.n_out * (p.swiglu ? 2 : 1) * p.k_in * 2;
  return bytes <= (int64_t)p.k_in * 48 * 1024 || (p.k_in >= 2048 && 3LL * p.rows <= p.E);
}

template <int DT, int ODT, bool SWIGLU>
hipError_t launch(const MmProblem& p, hipStream_t s) {
  const int numbers = p.rows / kRows + p.E;
  const bool by_row = p.rows < numbers;
  mm_narrow_kernel<DT, ODT, SWIGLU>
      <<<dim3(by_row ? p.rows : numbers, columns(p)), kWaves * 64, 0, s>>>(p, by_row);
  return hipGetLastError();
}

}  // namespace narrow

}  // namespace moe
