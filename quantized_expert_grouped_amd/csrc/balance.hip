// The router's load-balance loss, its per-expert counts and its gradient.  With p[t] = softmax of
// token t's E logits, n the valid tokens, c[e] how many of their K routes each went to expert e:
//   f[e] = c[e] / (n K),   P[e] = (1/n) sum_t p[t, e],   loss = E sum_e f[e] P[e],
//   d loss / d logits[t, j] = (E / n) p[t, j] (f[j] - sum_e f[e] p[t, e]),
// the counts being constants of the gradient.  Since sum_e p[t, e] = 1, f may be replaced by f -
// 1/E in the bracket, and is: near balance f is almost constant and the bracket a small difference
// of large terms otherwise.  f[e] - 1/E = (c[e] E - n K) / (E n K), exact integers up to one
// rounding.
//
// A row of logits is one wavefront's, read once into registers, the next row's loads under way
// meanwhile (-inf: an expert that the token may not take; a row of nothing else has p = 0).
// Forward: each workgroup keeps its rows' sums of p per column in registers and its counts in LDS
// and leaves one row of partial sums; a second launch adds those, and its last workgroup (an
// integer ticket) forms the loss.  All float sums are in an order that depends on the sizes and the
// valid rows alone.
//
// At E = 512 (us by the kernel trace, which adds a kernel's start): 8192 fp32 rows, forward 6.4, join
// 4.5, backward 7.5 (17 and 34 MB, 4.5 TB/s; starts and the waits of a row's reductions bound it);
// 30118 bf16 rows, a fifth of them invalid, 10.4, 4.5, 12.7 (backward, with its zero rows: 55 MB,
// 4.4 TB/s).  40 calls in one graph: forward with join 9.5 and 13.8, backward 6.6 and 12.0.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "mx.hpp"

namespace moe {

namespace {

constexpr int kWaves = 16;  // wavefronts of a workgroup
// of the backward pass, whose wavefronts share nothing (256 of 16: 500 rows 4.6 us instead of 2.7)
constexpr int kBackwardWaves = 4, kBackwardGroups = 1024;

// Workspace: ticket, each joining workgroup's part of the loss, then per workgroup valid tokens,
// counts [E], sums [E].
struct Partials {
  int32_t* ticket;
  float* loss;      // [kMaxJoins]
  int32_t* tokens;  // [kBalanceGroups]
  int32_t* counts;  // [groups x E]
  float* sums;      // [groups x E]
};
constexpr int kJoinCols = 32, kMaxJoins = 64;
static_assert((1 + kMaxJoins + kBalanceGroups) * 4 <= kBalanceHeader, "header");
__device__ __forceinline__ Partials partials(void* ws, int groups, int E) {
  Partials q;
  q.ticket = static_cast<int32_t*>(ws);
  q.loss = reinterpret_cast<float*>(q.ticket + 1);
  q.tokens = q.ticket + 1 + kMaxJoins;
  q.counts = q.ticket + kBalanceHeader / 4;
  q.sums = reinterpret_cast<float*>(q.counts + (size_t)groups * E);
  return q;
}

// The wavefront's largest value, or sum: DPP steps leave each row of 16 lanes with its row's, then
// the four rows' are read into scalars.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <class F>
__device__ __forceinline__ float wave_reduce(float v, F f) {
  v = f(v, dpp<0xB1>(v));   // quad_perm [1, 0, 3, 2]
  v = f(v, dpp<0x4E>(v));   // quad_perm [2, 3, 0, 1]
  v = f(v, dpp<0x141>(v));  // lane i <-> 7 - i within each half row
  v = f(v, dpp<0x140>(v));  // lane i <-> 15 - i within each row
  auto row = [&](int i) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * i));
  };
  return f(f(row(0), row(1)), f(row(2), row(3)));
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}

constexpr float kLog2E = 1.44269504088896341f;

// A lane's VPL columns of a row: VEC neighbours, then VEC neighbours 64 VEC further on, ...
template <int VEC>
__device__ __forceinline__ int column(int j, int lane) {
  return (j / VEC * 64 + lane) * VEC + j % VEC;
}

template <int DT, int VPL, int VEC>
struct Row {
  typedef typename Elem<DT>::type T;
  typedef T vec __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
  vec v[VPL / VEC];

  // columns past E stay at -inf: load leaves them alone
  __device__ __forceinline__ Row() {
#pragma unroll
    for (int j = 0; j < VPL; ++j) v[j / VEC][j % VEC] = (T)-INFINITY;
  }
  // E is a multiple of VEC; the row starts at any element (a wide load need not be aligned)
  __device__ __forceinline__ void load(const void* logits, int64_t at, int E, int lane) {
    const T* l = static_cast<const T*>(logits) + at;
#pragma unroll
    for (int i = 0; i < VPL / VEC; ++i) {
      const int c = column<VEC>(i * VEC, lane);
      if (c < E) v[i] = *reinterpret_cast<const vec*>(l + c);
    }
  }
  // exp(x - max) of each column times a factor near 1 that the row shares, 0 past E; returns 1 /
  // their sum, or 0 for a row with nothing above -inf.  The exponential is the hardware's 2^t of t =
  // x log2 e - c in one fma, c = max log2 e rounded once for the whole row (its rounding, below
  // 2^-8, is the factor).  So of a probability's error |x - max| 2^-24 is t's one rounding and a
  // quarter of that the constant's, besides 2^t's ulp; forming x - max first would round twice.  From
  // |max| = 2^16 on c's rounding could carry 2^t out of range, and x - max is formed first.  (With expf
  // the kernels were bound by its instructions.)  The maximum keeps a NaN, so a row that holds one, or
  // +inf, is NaN throughout and not taken for one with nothing above -inf.
  __device__ __forceinline__ float softmax(float (&p)[VPL]) const {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      p[j] = (float)v[j / VEC][j % VEC];
      m = __builtin_elementwise_maximum(m, p[j]);
    }
    m = wave_max(m);
    const bool none = m == -INFINITY;
    float s = 0.0f;
    if (fabsf(m) < 65536.0f) {  // uniform
      const float c = m * kLog2E;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        p[j] = __builtin_amdgcn_exp2f(fmaf(p[j], kLog2E, -c));
        s += p[j];
      }
    } else {
      const float from = none ? 0.0f : m;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        p[j] = __builtin_amdgcn_exp2f((p[j] - from) * kLog2E);
        s += p[j];
      }
    }
    s = wave_sum(s);
    const float r = __builtin_amdgcn_rcpf(s);  // 1 ulp; a Newton step leaves little more than half
    return none ? 0.0f : fmaf(r, fmaf(-s, r, 1.0f), r);
  }
};

// Bit l: row t + l * step is there and valid.  64 rows of a wavefront in one load: with a load per
// row, which the row's own has to wait for, its latency was a row's longest part.  t and step are
// uniform; t + 64 * step stays far below 2^31.
__device__ __forceinline__ uint64_t valid_rows(const BalanceArgs& a, int t, int step, int lane) {
  const int u = t + lane * step;
  bool on = u < a.T;
  if (on && a.valid) on = a.valid[u] != 0;
  return ballot(on);
}

template <int DT, int VPL, int VEC>
__global__ __launch_bounds__(kWaves * 64) void balance_rows_kernel(BalanceArgs a, void* ws) {
  constexpr int kCols = VPL * 64;
  __shared__ int32_t hist[kCols];
  __shared__ float half[kWaves / 2][kCols];
  __shared__ int32_t tokens;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Partials q = partials(ws, gridDim.x, a.E);
  const int step = gridDim.x * kWaves;
  int first = blockIdx.x * kWaves + wave;
  uint64_t left = valid_rows(a, first, step, lane);
  auto next_row = [&]() {  // the next valid row, or T
    while (left == 0 && first + 64 * step < a.T) {
      first += 64 * step;
      left = valid_rows(a, first, step, lane);
    }
    const int u = left ? first + __builtin_ctzll(left) * step : a.T;
    left &= left - 1;
    return u;
  };
  Row<DT, VPL, VEC> row;
  int32_t id = -1;
  auto fetch = [&](int u) {
    if (u < a.T) {
      row.load(a.logits, u * a.ld, a.E, lane);
      if (lane < a.K) id = a.idx[(int64_t)u * a.K + lane];
    }
  };
  int t = next_row();
  fetch(t);
  for (int e = threadIdx.x; e < kCols; e += kWaves * 64) hist[e] = 0;
  if (threadIdx.x == 0) {
    tokens = 0;
    if (blockIdx.x == 0) *q.ticket = 0;
  }
  __syncthreads();
  float acc[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) acc[j] = 0.0f;
  int mine = 0;
  while (t < a.T) {
    const Row<DT, VPL, VEC> now = row;
    const int32_t e = id;
    t = next_row();
    fetch(t);
    ++mine;
    if (lane < a.K && e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
    float p[VPL];
    const float r = now.softmax(p);
#pragma unroll
    for (int j = 0; j < VPL; ++j) acc[j] = fmaf(p[j], r, acc[j]);
  }
  if (lane == 0 && mine) atomicAdd(&tokens, mine);
  // the wavefronts' sums, the upper half onto the lower until one is left
#pragma unroll
  for (int n = kWaves / 2; n >= 1; n /= 2) {
    if (wave >= n && wave < 2 * n)
#pragma unroll
      for (int j = 0; j < VPL; ++j) half[wave - n][j * 64 + lane] = acc[j];
    __syncthreads();
    if (wave < n)
#pragma unroll
      for (int j = 0; j < VPL; ++j) acc[j] += half[wave][j * 64 + lane];
    __syncthreads();
  }
  if (wave == 0)
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = column<VEC>(j, lane);
      if (c < a.E) q.sums[(size_t)blockIdx.x * a.E + c] = acc[j];
    }
  for (int e = threadIdx.x; e < a.E; e += kWaves * 64)
    q.counts[(size_t)blockIdx.x * a.E + e] = hist[e];
  if (threadIdx.x == 0) q.tokens[blockIdx.x] = tokens;
}

// 32 columns by 32 strands of workgroups' partial rows, 8 of them each, all loads under way at
// once.
__global__ __launch_bounds__(1024) void balance_join_kernel(int E, int K, int groups, void* ws,
                                                            int32_t* __restrict__ counts,
                                                            float* __restrict__ prob_mean,
                                                            float* __restrict__ loss) {
  constexpr int kStrands = 32;
  static_assert(kBalanceGroups == 8 * kStrands, "8 rows a strand");
  __shared__ int32_t cs[16][kJoinCols];
  __shared__ float ss[16][kJoinCols];
  __shared__ int32_t ns[4];
  const Partials q = partials(ws, groups, E);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int e = blockIdx.x * kJoinCols + col;
  int32_t c8[8];
  float s8[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int g = strand + kStrands * i;
    const bool on = g < groups && e < E;
    c8[i] = on ? q.counts[(size_t)g * E + e] : 0;
    s8[i] = on ? q.sums[(size_t)g * E + e] : 0.0f;
  }
  int n = threadIdx.x < groups ? q.tokens[threadIdx.x] : 0;  // the first 256 threads
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o);
  if (lane == 0 && wave < 4) ns[wave] = n;
  int32_t c = ((c8[0] + c8[1]) + (c8[2] + c8[3])) + ((c8[4] + c8[5]) + (c8[6] + c8[7]));
  float s = ((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7]));
  c += __shfl_xor(c, 32);  // the wavefront's two strands
  s += __shfl_xor(s, 32);
  if (lane < 32) {
    cs[wave][col] = c;
    ss[wave][col] = s;
  }
  __syncthreads();
  n = (ns[0] + ns[1]) + (ns[2] + ns[3]);
  if (wave == 0) {
    c = 0;
    s = 0.0f;
    if (lane < 32)
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        c += cs[w][col];
        s += ss[w][col];
      }
    const float mean = n > 0 ? s / (float)n : 0.0f;
    if (lane < 32 && e < E) {
      counts[e] = c;
      prob_mean[e] = mean;
    }
    const float part = wave_sum((float)c * mean);  // 0 in lanes without a column
    int before = 0;
    if (lane == 0) {
      if (blockIdx.x == 0) counts[E] = n;
      __hip_atomic_store(q.loss + blockIdx.x, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      before = __hip_atomic_fetch_add(q.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(before) != (int)gridDim.x - 1) return;
    const float v = lane < (int)gridDim.x ? __hip_atomic_load(q.loss + lane, __ATOMIC_RELAXED,
                                                              __HIP_MEMORY_SCOPE_AGENT)
                                          : 0.0f;
    const float sum = wave_sum(v);
    if (lane == 0) *loss = n > 0 ? sum * ((float)E / ((float)n * (float)K)) : 0.0f;
  }
}

constexpr int kWaitLoads = 0x0f70;  // s_waitcnt vmcnt(0)
template <int DT, int VPL, int VEC>
__global__ __launch_bounds__(kBackwardWaves * 64) void balance_backward_kernel(
    BalanceArgs a, const int32_t* __restrict__ counts, const float* __restrict__ grad_loss,
    void* __restrict__ grad, int64_t ld_grad) {
  typedef Row<DT, VPL, VEC> R;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int step = gridDim.x * kBackwardWaves;
  int t = blockIdx.x * kBackwardWaves + wave, i64 = 0;
  uint64_t valid = valid_rows(a, t, step, lane);
  R row;
  bool on = false;
  auto fetch = [&]() {
    on = t < a.T && (valid >> i64 & 1);
    if (on) row.load(a.logits, t * a.ld, a.E, lane);
  };
  fetch();
  const int n = counts[a.E];
  typedef int32_t ivec __attribute__((ext_vector_type(VEC), aligned(4)));
  ivec c[VPL / VEC];
#pragma unroll
  for (int i = 0; i < VPL / VEC; ++i) {
    c[i] = (ivec)0;
    if (column<VEC>(i * VEC, lane) < a.E)
      c[i] = *reinterpret_cast<const ivec*>(counts + column<VEC>(i * VEC, lane));
  }
  // g (E / n) (f - 1/E) = g (c E - n K) / (n n K); below 2^53, so exact in fp64, whose one fma takes
  // an eighth of the 64-bit integers' instructions
  const float nf = (float)n;
  const float scale =
      n > 0 ? (grad_loss ? *grad_loss : 1.0f) / (nf * (float)a.K) / nf : 0.0f;
  float dev[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    dev[j] = (float)fma((double)c[j / VEC][j % VEC], (double)a.E, -((double)n * a.K)) * scale;
  while (t < a.T) {
    const R now = row;
    const bool live = on;
    typename R::T* g = static_cast<typename R::T*>(grad) + t * ld_grad;
    t += step;
    i64 = (i64 + 1) & 63;
    if (i64 == 0 && t < a.T) valid = valid_rows(a, t, step, lane);
    fetch();
    float y[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) y[j] = 0.0f;
    if (live) {
      const float r = now.softmax(y);
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) dot = fmaf(y[j], dev[j], dot);
      dot = wave_sum(dot) * r;
#pragma unroll
      for (int j = 0; j < VPL; ++j) y[j] = y[j] * r * (dev[j] - dot);
    }
    // the next row's loads before the stores, which would be waited for with them otherwise
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
#pragma unroll
    for (int i = 0; i < VPL / VEC; ++i) {
      const int e = column<VEC>(i * VEC, lane);
      typedef float fvec __attribute__((ext_vector_type(VEC)));
      fvec f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = y[i * VEC + j];
      if (e < a.E)
        *reinterpret_cast<typename R::vec*>(g + e) = __builtin_convertvector(f, typename R::vec);
    }
  }
}

// VEC values of a row are loaded together, 16 bytes at most, where E allows it, from any element's
// address: which columns a lane sums, and with it the order of the sums, goes by E alone.  (30118
// bf16 rows of 512, 513 apart: forward and join 14.1 us, backward 11.4, as with aligned rows; with
// single values 15.1 and 13.5.)
template <int DT, class F>
hipError_t dispatch(int E, F f) {
  constexpr int kMost = DT == kF32 ? 4 : 8;
  const int vpl = (E + 63) / 64;
  auto go = [&](auto V) {
    constexpr int VPL = decltype(V)::value;
    constexpr int VEC = VPL < kMost ? VPL : kMost;
    if (E % VEC == 0)
      f(V, std::integral_constant<int, VEC>{});
    else
      f(V, std::integral_constant<int, 1>{});
    return hipGetLastError();
  };
  return vpl <= 1    ? go(std::integral_constant<int, 1>{})
         : vpl <= 2  ? go(std::integral_constant<int, 2>{})
         : vpl <= 4  ? go(std::integral_constant<int, 4>{})
         : vpl <= 8  ? go(std::integral_constant<int, 8>{})
         : vpl <= 16 ? go(std::integral_constant<int, 16>{})
                     : go(std::integral_constant<int, 32>{});
}

template <int DT>
hipError_t forward(const BalanceArgs& a, void* ws, hipStream_t s) {
  return dispatch<DT>(a.E, [&](auto V, auto W) {
    balance_rows_kernel<DT, decltype(V)::value, decltype(W)::value>
        <<<balance_groups(a.T), kWaves * 64, 0, s>>>(a, ws);
  });
}

template <int DT>
hipError_t backward(const BalanceArgs& a, const int32_t* counts, const float* grad_loss, void* grad,
                    int64_t ld, hipStream_t s) {
  const int groups = (a.T + kBackwardWaves - 1) / kBackwardWaves;
  return dispatch<DT>(a.E, [&](auto V, auto W) {
    balance_backward_kernel<DT, decltype(V)::value, decltype(W)::value>
        <<<groups < kBackwardGroups ? groups : kBackwardGroups, kBackwardWaves * 64, 0, s>>>(
            a, counts, grad_loss, grad, ld);
  });
}

}  // namespace

hipError_t launch_balance_loss(const BalanceArgs& a, int32_t* counts, float* prob_mean, float* loss,
                               void* ws, hipStream_t s) {
  hipError_t e = a.dtype == kF32    ? forward<kF32>(a, ws, s)
                 : a.dtype == kBF16 ? forward<kBF16>(a, ws, s)
                                    : forward<kF16>(a, ws, s);
  if (e != hipSuccess) return e;
  balance_join_kernel<<<(a.E + kJoinCols - 1) / kJoinCols, 1024, 0, s>>>(
      a.E, a.K, balance_groups(a.T), ws, counts, prob_mean, loss);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, const int32_t* counts,
                                   const float* grad_loss, void* grad, int64_t ld_grad,
                                   hipStream_t s) {
  return a.dtype == kF32    ? backward<kF32>(a, counts, grad_loss, grad, ld_grad, s)
         : a.dtype == kBF16 ? backward<kBF16>(a, counts, grad_loss, grad, ld_grad, s)
                            : backward<kF16>(a, counts, grad_loss, grad, ld_grad, s);
}

}  // namespace moe
