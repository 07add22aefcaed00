// The grouped product of 16-bit rows and weights, and its gradients.  All three are sums of
// products over one index,
//   forward  y[r, n]     = sum_k a[a(r), k] w[e, n, k]
//   dgrad    da[r, k]    = sum_n grad[r, n] w[e, n, k]
//   wgrad    dw[e, n, k] = sum_r grad[r, n] a[a(r), k]
// and run as D[i, j] = sum_c P[i, c] Q[j, c] on the matrix cores, where i is the index that is
// contiguous in the result: P is w, w transposed, a transposed, and Q is a, grad, grad transposed.
// Sums are in fp32, in an order that depends on the sizes alone.
#include "mm.hpp"

namespace moe {

namespace {

constexpr int kBlockI = 64, kBlockJ = 128, kBlockC = 32, kPitch = kBlockC + 8;

// Rows of an expert: tiles of kBlockJ rows are numbered offsets[e] / kBlockJ + e and on, which
// leaves room for all of them and grows from expert to expert; some numbers belong to no tile.
struct Rows {
  int expert, row0, nrows;
};
__device__ __forceinline__ Rows find_rows(const MmProblem& p, int id) {
  const int lane = threadIdx.x & 63;
  int upto = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    const int e = e0 + lane;
    upto += __popcll(ballot(e < p.E && p.offsets[min(e, p.E)] / kBlockJ + e <= id));
  }
  Rows t;
  t.expert = max(upto - 1, 0);
  const int first = p.offsets[t.expert], last = min(p.offsets[t.expert + 1], p.rows);
  t.row0 = first + (id - (first / kBlockJ + t.expert)) * kBlockJ;
  t.nrows = min(last - t.row0, kBlockJ);
  return t;
}

// A tile of 64 i by 128 j, a wavefront 64 x 32 of it; operands go through registers into LDS.
// SwiGLU's forward takes 32 gates and their 32 ups as its i.
template <int OP, int DT, int ODT, bool SWIGLU>
__global__ __launch_bounds__(256) void mm_kernel(MmProblem p) {
  typedef typename Half<DT>::T T;
  typedef typename Half<DT>::v8 v8;
  constexpr bool kGates = OP == kMmForward && SWIGLU;
  __shared__ alignas(16) T ps[kBlockI][kPitch], qs[kBlockJ][kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  int e, row0, nrows, j0 = 0, i0;
  if constexpr (OP == kMmWgrad) {
    e = blockIdx.x;
    row0 = min(p.offsets[e], p.rows);
    nrows = max(min(p.offsets[e + 1], p.rows) - row0, 0);
    j0 = blockIdx.y * kBlockJ;
    i0 = blockIdx.z * kBlockI;
  } else {
    const Rows t = find_rows(p, blockIdx.x);
    if (t.nrows <= 0) return;
    e = t.expert, row0 = t.row0, nrows = t.nrows;
    i0 = blockIdx.y * (kGates ? 32 : 64);
  }
  const int ni = OP == kMmForward ? p.n_out : p.k_in;                           // i's
  const int nj = OP == kMmWgrad ? p.n_out : nrows;                              // j's
  const int nc = OP == kMmForward ? p.k_in : OP == kMmDgrad ? p.n_out : nrows;  // c's
  const int mat_rows = kGates ? 2 * p.n_out : p.n_out;
  const T* w = static_cast<const T*>(p.w) + (int64_t)e * mat_rows * p.k_in;
  const T* a = static_cast<const T*>(p.a);
  const T* g = static_cast<const T*>(p.grad);
  const v8 zero = {};

  v16f acc[2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[m][q] = 0.0f;
  for (int c0 = 0; c0 < nc; c0 += kBlockC) {
    __syncthreads();
    {  // P: 64 x 32
      if constexpr (OP == kMmForward) {
        const int i = threadIdx.x >> 2, c = c0 + (threadIdx.x & 3) * 8;
        const int n = kGates ? (i < 32 ? i0 + i : p.n_out + i0 + i - 32) : i0 + i;
        const bool on = c < nc && (kGates ? i0 + (i & 31) : n) < ni;
        *reinterpret_cast<v8*>(&ps[i][c - c0]) =
            on ? *reinterpret_cast<const v8*>(w + (int64_t)n * p.k_in + c) : zero;
      } else {
        const int c = c0 + (threadIdx.x >> 3), i = (threadIdx.x & 7) * 8;
        v8 v = zero;
        if (c < nc && i0 + i < ni)
          v = *reinterpret_cast<const v8*>(
              OP == kMmDgrad ? w + (int64_t)c * p.k_in + i0 + i
                             : a + act_row(p, row0 + c) * p.lda + i0 + i);
#pragma unroll
        for (int q = 0; q < 8; ++q) ps[i + q][c - c0] = v[q];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // Q: 128 x 32
      const int t = threadIdx.x + 256 * h;
      if constexpr (OP == kMmWgrad) {
        const int c = c0 + (t >> 4), j = (t & 15) * 8;
        v8 v = zero;
        if (c < nc && j0 + j < nj)
          v = *reinterpret_cast<const v8*>(g + (int64_t)(row0 + c) * p.ldg + j0 + j);
#pragma unroll
        for (int q = 0; q < 8; ++q) qs[j + q][c - c0] = v[q];
      } else {
        const int j = t >> 2, c = c0 + (t & 3) * 8;
        v8 v = zero;
        if (c < nc && j < nj)
          v = *reinterpret_cast<const v8*>(OP == kMmForward
                                               ? a + act_row(p, row0 + j) * p.lda + c
                                               : g + (int64_t)(row0 + j) * p.ldg + c);
        *reinterpret_cast<v8*>(&qs[j][c - c0]) = v;
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kBlockC; c += 16) {
      const v4i q = *reinterpret_cast<const v4i*>(&qs[32 * wave + (lane & 31)][c + 8 * half]);
#pragma unroll
      for (int m = 0; m < 2; ++m)
        acc[m] = mfma16<DT>(
            *reinterpret_cast<const v4i*>(&ps[32 * m + (lane & 31)][c + 8 * half]), q, acc[m]);
    }
  }
  const int j = j0 + 32 * wave + (lane & 31);
  if (j >= nj) return;
#pragma unroll
  for (int m = 0; m < (kGates ? 1 : 2); ++m)
#pragma unroll
    for (int q = 0; q < 16; q += 4) {
      const int i = i0 + 32 * m + 2 * q + 4 * half;
      if (i >= ni) continue;
      const v4f y = {acc[m][q], acc[m][q + 1], acc[m][q + 2], acc[m][q + 3]};
      const v4f u = {acc[1][q], acc[1][q + 1], acc[1][q + 2], acc[1][q + 3]};
      if constexpr (OP == kMmForward)
        finish_forward<DT, ODT, SWIGLU>(p, e, row0 + j, i, y, u);
      else if constexpr (OP == kMmDgrad)
        finish_dgrad<DT, ODT, SWIGLU>(p, row0 + j, i, y);
      else
        store4<ODT>(p.out, ((int64_t)e * p.n_out + j) * p.k_in + i, y);
    }
}

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

template <int OP, int DT, int ODT, bool SWIGLU>
hipError_t launch(const MmProblem& p, hipStream_t s) {
  const int ni = OP == kMmForward ? p.n_out : p.k_in;
  const int wide = OP == kMmForward && SWIGLU ? 32 : 64;
  dim3 grid(p.rows / kBlockJ + p.E, (ni + wide - 1) / wide);
  if (OP == kMmWgrad) grid = dim3(p.E, (p.n_out + kBlockJ - 1) / kBlockJ, (ni + 63) / 64);
  mm_kernel<OP, DT, ODT, SWIGLU><<<grid, 256, 0, s>>>(p);
  if (OP == kMmWgrad && p.bias_out)
    mm_bias_kernel<DT, ODT><<<dim3(p.E, (p.n_out + 255) / 256), 64, 0, s>>>(p);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_type(const MmProblem& p, hipStream_t s) {
  if (p.op == kMmForward)
    return p.swiglu            ? launch<kMmForward, DT, DT, true>(p, s)
           : p.out_dtype == DT ? launch<kMmForward, DT, DT, false>(p, s)
                               : launch<kMmForward, DT, kF32, false>(p, s);
  if (p.op == kMmDgrad)
    return p.swiglu            ? launch<kMmDgrad, DT, DT, true>(p, s)
           : p.out_dtype == DT ? launch<kMmDgrad, DT, DT, false>(p, s)
                               : launch<kMmDgrad, DT, kF32, false>(p, s);
  return p.out_dtype == DT ? launch<kMmWgrad, DT, DT, false>(p, s)
                           : launch<kMmWgrad, DT, kF32, false>(p, s);
}

}  // namespace

size_t mm_wgrad_workspace(int, int, int, int) { return 0; }

hipError_t launch_mm(const MmProblem& p_, void*, hipStream_t s) {
  MmProblem p = p_;
  // n / K = n * k_mul >> k_shift for n < 2^30, K <= 64
  p.k_shift = 30;
  while (1 << (p.k_shift - 30) < p.K) ++p.k_shift;
  p.k_mul = (uint32_t)(((uint64_t)1 << p.k_shift) / p.K + 1);
  return p.dtype == kBF16 ? launch_type<kBF16>(p, s) : launch_type<kF16>(p, s);
}

}  // namespace moe
