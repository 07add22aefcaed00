// Rows to MXFP4 and back (the format and its rounding: mx.hpp).
//
// Both kernels move each byte once and are bound by memory.  A lane owns 8 values: 16 or 32 bytes
// in, one dword of codes, so a block of 32 is a quad of lanes whose largest magnitude takes two DPP
// steps.  8192 x 2048 values: fp32 quantised in 11 to 12 us (76 MB, 6.4 TB/s, partly
// from the caches), dequantised to bf16 in 9 to 11 us (42 MB, 4.2 TB/s).
#include "mx.hpp"

namespace moe {

namespace {

constexpr int kDppXor1 = 0xB1;  // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;  // quad_perm [2, 3, 0, 1]

#define quad(v, ctrl) \
  __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xF, 0xF, false))

template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&v)[8]) {
  if constexpr (DT == kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    typedef typename Elem<DT>::type T;
    typedef T v8 __attribute__((ext_vector_type(8)));
    const v8 a = *reinterpret_cast<const v8*>(static_cast<const T*>(base) + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
  }
}

template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, int64_t ldx,
                                                          int64_t n, uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const int64_t row = blockIdx.y;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= n) return;  // whole quads: n is a multiple of 32
  float v[8];
  load8<DT>(x, row * ldx + i, v);
  float m = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = mx_amax(m, v[j]);
  m = mx_amax(m, quad(m, kDppXor1));
  m = mx_amax(m, quad(m, kDppXor2));
  const uint32_t byte = mx_scale_byte(m);
  const uint32_t w = mx_codes8(v, byte);
  const int64_t at = row * n + i;
  *reinterpret_cast<uint32_t*>(codes + at / 2) = w;
  if ((threadIdx.x & 3) == 0) scales[at / kMxBlock] = (uint8_t)byte;
}

// code -> its value times the block's scale
__device__ __forceinline__ float mx_value(uint32_t code, float scale) {
  const uint32_t e = (code >> 1) & 3u, mant = code & 1u;
  const float mag =
      e == 0 ? 0.5f * (float)mant : __uint_as_float(((e + 126u) << 23) | (mant << 22));
  return ((code & 8u) ? -mag : mag) * scale;
}

template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            int64_t n, void* __restrict__ y,
                                                            int64_t ldy) {
  const int64_t row = blockIdx.y;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  const int64_t at = row * n + i;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + at / 2);
  const uint32_t byte = scales[at / kMxBlock];
  const float scale = byte == 255u ? __uint_as_float(0x7fc00000u)
                      : byte == 0u ? __uint_as_float(0x00400000u)  // 2^-127, subnormal
                                   : __uint_as_float(byte << 23);
  typedef typename Elem<DT>::type T;
  constexpr int N = 16 / sizeof(T);  // values of a 16-byte store
  typedef T vec __attribute__((ext_vector_type(N)));
  vec* p = reinterpret_cast<vec*>(static_cast<T*>(y) + row * ldy + i);
#pragma unroll
  for (int h = 0; h < 8 / N; ++h) {
    vec v;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = (T)mx_value((w >> (4 * (h * N + j))) & 15u, scale);
    p[h] = v;
  }
}

// Rows that follow each other without a gap are one row, as long as its workgroups of 2048 values
// fit a grid's x.
inline void collapse(int64_t ld, int64_t& rows, int64_t& n) {
  if (ld == n && rows * n <= (int64_t)1 << 33) {
    n *= rows;
    rows = 1;
  }
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int dtype, int64_t ldx, int rows_, int n_,
                              uint8_t* codes, uint8_t* scales, hipStream_t s) {
  int64_t rows = rows_, n = n_;
  collapse(ldx, rows, n);
  for (int64_t r0 = 0; r0 < rows; r0 += 65535) {  // a grid's largest y
    const int64_t k = rows - r0 < 65535 ? rows - r0 : 65535;
    const dim3 grid((unsigned)((n / 8 + 255) / 256), (unsigned)k);
    const char* xr = static_cast<const char*>(x) + r0 * ldx * (dtype == kF32 ? 4 : 2);
    uint8_t* c = codes + r0 * n / 2;
    uint8_t* b = scales + r0 * n / kMxBlock;
    if (dtype == kF32)
      mx_quantize_kernel<kF32><<<grid, 256, 0, s>>>(xr, ldx, n, c, b);
    else if (dtype == kBF16)
      mx_quantize_kernel<kBF16><<<grid, 256, 0, s>>>(xr, ldx, n, c, b);
    else
      mx_quantize_kernel<kF16><<<grid, 256, 0, s>>>(xr, ldx, n, c, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int rows_, int n_,
                                void* y, int dtype, int64_t ldy, hipStream_t s) {
  int64_t rows = rows_, n = n_;
  collapse(ldy, rows, n);
  for (int64_t r0 = 0; r0 < rows; r0 += 65535) {
    const int64_t k = rows - r0 < 65535 ? rows - r0 : 65535;
    const dim3 grid((unsigned)((n / 8 + 255) / 256), (unsigned)k);
    char* yr = static_cast<char*>(y) + r0 * ldy * (dtype == kF32 ? 4 : 2);
    const uint8_t* c = codes + r0 * n / 2;
    const uint8_t* b = scales + r0 * n / kMxBlock;
    if (dtype == kF32)
      mx_dequantize_kernel<kF32><<<grid, 256, 0, s>>>(c, b, n, yr, ldy);
    else
      mx_dequantize_kernel<kBF16><<<grid, 256, 0, s>>>(c, b, n, yr, ldy);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
