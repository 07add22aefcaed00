// The grouped MXFP4 product: row r of expert e is
//   y[r, n] = sum over blocks b of 2^(ea - 127) 2^(ew - 127) sum_j A[row(r), 32 b + j] W[e, n, 32 b + j],
// which v_mfma_scale_f32_32x32x64_f8f6f4 computes whole: e2m1 codes and the blocks' scale bytes go
// in as they lie in memory, sums stay in fp32.
//
// Operands: the weights are the MFMA's A (its rows are output columns n), the activations its B (its
// columns are routed rows), so a lane's 16 results are 4 runs of 4 consecutive n of one routed
// row.  Lane l of an operand holds one block of one row: row l % 32 and, of the MFMA's two blocks, l / 32,
// as 16 bytes of codes and one scale byte (a byte of a register that the instruction picks).  The order
// in which blocks are taken is free as long as both operands agree, so a lane takes runs of
// consecutive blocks.
#include "common.hpp"
#include "mx.hpp"

namespace moe {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;  // the instruction's format code of e2m1

template <int SEL>
__device__ __forceinline__ v16f mfma_mx(const v4i& w, const v4i& a, const v16f& c, int sw, int sa) {
  const v8i w8 = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, a8, c, kFp4, kFp4, SEL, sw, SEL, sa);
}

// The expert whose tile `id` is, and the tile's rows.  Tiles of BM rows are numbered without a pass
// over the experts' counts: expert e's start at offsets[e] / BM + e, which leaves room for all of
// them (ceil(n / BM) <= (offsets[e] + n) / BM - offsets[e] / BM + 1) and grows by one at least
// from expert to expert, so a tile's expert is the last one whose first number is not above it.
// Some numbers belong to no tile: those workgroups end.  With fewer rows than that gives numbers, a tile is
// numbered by its first row instead (`by_row`).  Two rounds of 64 lanes search 2048 experts.
struct Tile {
  int expert, row0, nrows;
};
template <int BM>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ offsets, int E, int rows, int id,
                                          bool by_row) {
  const int lane = threadIdx.x & 63;
  auto key = [&](int e) { return by_row ? offsets[e] : offsets[e] / BM + e; };
  const int step = (E + 63) / 64;
  const int c1 = __popcll(ballot(lane * step < E && key(min(lane * step, E - 1)) <= id));
  const int seg = max(c1 - 1, 0) * step;
  const int c2 = __popcll(ballot(lane < step && seg + lane < E && key(min(seg + lane, E - 1)) <= id));
  Tile t;
  t.expert = seg + max(c2 - 1, 0);
  const int first = offsets[t.expert];
  const int last = min(offsets[t.expert + 1], rows);
  if (by_row) {
    t.row0 = id;
    if ((id - first) % BM != 0 || id < first) t.row0 = last;
  } else {
    t.row0 = first + (id - key(t.expert)) * BM;
  }
  t.nrows = min(last - t.row0, BM);  // <= 0: no tile
  return t;
}

// silu(g) * u in fp32; g far below zero gives g / inf = -0
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// ---- few rows ------------------------------------------------------------------------------
// One workgroup: up to 32 rows of an expert by 32 columns (SwiGLU: 32 gates and their 32 ups), K
// split over its 4 wavefronts and joined in LDS.
template <int EPI>
__global__ __launch_bounds__(256) void mx_mm_narrow_kernel(MxProblem p, bool by_row) {
  constexpr int kMats = EPI == kMxSwiglu ? 2 : 1;
  __shared__ float part[4][kMats][32][36];
  const Tile t = find_tile<32>(p.offsets, p.E, p.rows, blockIdx.x, by_row);
  if (t.nrows <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int half = lane >> 5, l32 = lane & 31;
  const int n0 = blockIdx.y * 32;
  const size_t kb = p.k_in / 2, sb = p.k_in / kMxBlock;
  int r = t.row0 + min(l32, t.nrows - 1);
  if (p.src) r = p.src[r] / p.K;
  r = min(max(r, 0), p.n_act - 1);
  const uint8_t* a = p.a + (size_t)r * kb + 32 * half;
  const uint8_t* as = p.as + (size_t)r * sb + 2 * half;
  const size_t wrow = (size_t)t.expert * p.n_out * kMats + n0 + l32;
  const uint8_t* w = p.w + wrow * kb + 32 * half;
  const uint8_t* ws = p.ws + wrow * sb + 2 * half;
  const size_t up = (size_t)p.n_out;  // rows from a gate to its up

  v16f acc[kMats];
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[m][i] = 0.0f;

  for (int c = wave; c < p.k_in / 128; c += 4) {
    const v4i a0 = *reinterpret_cast<const v4i*>(a + c * 64);
    const v4i a1 = *reinterpret_cast<const v4i*>(a + c * 64 + 16);
    const int sa = *reinterpret_cast<const uint16_t*>(as + c * 4);
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      const uint8_t* wm = w + m * up * kb + c * 64;
      const v4i w0 = *reinterpret_cast<const v4i*>(wm);
      const v4i w1 = *reinterpret_cast<const v4i*>(wm + 16);
      const int sw = *reinterpret_cast<const uint16_t*>(ws + m * up * sb + c * 4);
      acc[m] = mfma_mx<0>(w0, a0, acc[m], sw, sa);
      acc[m] = mfma_mx<1>(w1, a1, acc[m], sw, sa);
    }
  }
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<float4*>(&part[wave][m][l32][2 * i + 4 * half]) =
          make_float4(acc[m][i], acc[m][i + 1], acc[m][i + 2], acc[m][i + 3]);
  __syncthreads();

  // thread: row tr, 4 columns
  const int tr = threadIdx.x >> 3, tc = (threadIdx.x & 7) * 4;
  float y[kMats][4];
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[m][j] = (part[0][m][tr][tc + j] + part[1][m][tr][tc + j]) +
                (part[2][m][tr][tc + j] + part[3][m][tr][tc + j]);
  const size_t row = (size_t)t.row0 + tr;
  const bool live = tr < t.nrows;
  if constexpr (EPI == kMxSwiglu) {
    float h[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = swiglu(y[0][j], y[1][j]);
      h[j + 4] = 0.0f;
      m = max(m, __float_as_uint(h[j]) & 0x7fffffffu);
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    m = max(m, (uint32_t)__shfl_xor((int)m, 4));
    const uint32_t byte = mx_scale_byte(m);
    const float inv = mx_inverse_scale(byte);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] *= inv;
    const uint32_t codes = byte == 255u ? 0u : mx_codes8(h);
    if (live) {
      uint8_t* o = static_cast<uint8_t*>(p.out) + row * (p.n_out / 2) + (n0 + tc) / 2;
      *reinterpret_cast<uint16_t*>(o) = (uint16_t)codes;
      if ((threadIdx.x & 7) == 0) p.out_scales[row * (p.n_out / kMxBlock) + n0 / kMxBlock] = (uint8_t)byte;
    }
  } else if (live) {
    if constexpr (EPI == kMxF32) {
      float* o = static_cast<float*>(p.out) + row * p.n_out + n0 + tc;
      *reinterpret_cast<float4*>(o) = make_float4(y[0][0], y[0][1], y[0][2], y[0][3]);
    } else {
      typedef __bf16 v4 __attribute__((ext_vector_type(4)));
      __bf16* o = static_cast<__bf16*>(p.out) + row * p.n_out + n0 + tc;
      *reinterpret_cast<v4*>(o) = (v4){(__bf16)y[0][0], (__bf16)y[0][1], (__bf16)y[0][2], (__bf16)y[0][3]};
    }
  }
}

}  // namespace

hipError_t launch_mx_mm(const MxProblem& p, hipStream_t s) {
  const int numbers = p.rows / 32 + p.E;
  const bool by_row = p.rows < numbers;
  const dim3 grid((unsigned)(by_row ? p.rows : numbers), (unsigned)(p.n_out / 32));
  if (p.epilogue == kMxF32)
    mx_mm_narrow_kernel<kMxF32><<<grid, 256, 0, s>>>(p, by_row);
  else if (p.epilogue == kMxBF16)
    mx_mm_narrow_kernel<kMxBF16><<<grid, 256, 0, s>>>(p, by_row);
  else
    mx_mm_narrow_kernel<kMxSwiglu><<<grid, 256, 0, s>>>(p, by_row);
  return hipGetLastError();
}

}  // namespace moe
