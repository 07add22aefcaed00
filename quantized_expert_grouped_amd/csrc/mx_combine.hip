// Combine of bf16 expert rows ("#1282 prefill: STRATA_PREFILL_CPU_SHARE=auto hands a small chunk's
// least-routed experts to the idle CPU pool", "What it does": Dm's rows are unweighted, the combine
// applies the routing weights):
//   out[t, i] = sum_{k < K} w[t, k] * rows[slot[t*K + k], i],
// k ascending, fp32 fused multiply-adds, each bf16 value widened exactly.  A route whose slot is no row (-1:
// its expert id was out of range) adds nothing.
#include "mx.hpp"

namespace moe {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

__global__ __launch_bounds__(256) void combine_bf16_kernel(const uint16_t* __restrict__ rows,
                                                           const int32_t* __restrict__ slot,
                                                           const float* __restrict__ w, int n_rows, int K,
                                                           int H, float* __restrict__ out) {
  const int t = blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 8;
  if (c >= H) return;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k = 0; k < K; ++k) {
    const int r = slot[(size_t)t * K + k];
    if ((uint32_t)r >= (uint32_t)n_rows) continue;  // uniform
    const float wk = w[(size_t)t * K + k];
    const v4u d = *reinterpret_cast<const v4u*>(rows + (size_t)r * H + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[2 * j] = fmaf(wk, __uint_as_float(d[j] << 16), acc[2 * j]);
      acc[2 * j + 1] = fmaf(wk, __uint_as_float(d[j] & 0xffff0000u), acc[2 * j + 1]);
    }
  }
  v4f* o = reinterpret_cast<v4f*>(out + (size_t)t * H + c);
  o[0] = (v4f){acc[0], acc[1], acc[2], acc[3]};
  o[1] = (v4f){acc[4], acc[5], acc[6], acc[7]};
}

}  // namespace

hipError_t launch_combine_bf16(const void* rows, const int32_t* slot, const float* w, int T, int K,
                               int H, float* out, hipStream_t s) {
  const dim3 grid(T, (H / 8 + 255) / 256);
  combine_bf16_kernel<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(rows), slot, w, T * K, K, H,
                                           out);
  return hipGetLastError();
}

}  // namespace moe
