// Combine of bf16 expert rows ("#1282 prefill: STRATA_PREFILL_CPU_SHARE=auto hands a small chunk's
// least-routed experts to the idle CPU pool", "What it does": Dm's rows are unweighted, the combine
// applies the routing weights):
//   out[t, i] = sum_{k < K} w[t, k] * rows[slot[t*K + k], i],
// k ascending, fp32 fused multiply-adds, each bf16 value widened exactly.  A route whose slot is no
// row (-1: its expert id was out of range) adds nothing.
#include "mx.hpp"

namespace moe {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

// A thread owns 8 columns of a token and keeps up to kBatch rows' loads under way (each row is read
// once: non-temporal); the token's slots and weights are scalars.  Bound by memory: 8192 tokens,
// K = 10, H = 2048 (403 MB) take 69 to 73 us, 5.5 to 5.9 TB/s; with one row's
// plain load at a time, 84.
constexpr int kBatch = 8;

__global__ __launch_bounds__(256) void combine_bf16_kernel(const uint16_t* __restrict__ rows,
                                                           const int32_t* __restrict__ slot,
                                                           const float* __restrict__ w, int n_rows,
                                                           int K, int H, float* __restrict__ out) {
  const int t = blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 8;
  if (c >= H) return;
  const int32_t* sl = slot + (size_t)t * K;
  const float* wt = w + (size_t)t * K;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k0 = 0; k0 < K; k0 += kBatch) {
    v4u d[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (k0 + j < K && (uint32_t)sl[k0 + j] < (uint32_t)n_rows)  // uniform
        d[j] = __builtin_nontemporal_load(
            reinterpret_cast<const v4u*>(rows + (size_t)sl[k0 + j] * H + c));
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (k0 + j < K && (uint32_t)sl[k0 + j] < (uint32_t)n_rows) {
        const float wk = wt[k0 + j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] = fmaf(wk, __uint_as_float(d[j][i] << 16), acc[2 * i]);
          acc[2 * i + 1] = fmaf(wk, __uint_as_float(d[j][i] & 0xffff0000u), acc[2 * i + 1]);
        }
      }
    }
  }
  v4f* o = reinterpret_cast<v4f*>(out + (size_t)t * H + c);
  __builtin_nontemporal_store((v4f){acc[0], acc[1], acc[2], acc[3]}, o);
  __builtin_nontemporal_store((v4f){acc[4], acc[5], acc[6], acc[7]}, o + 1);
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
