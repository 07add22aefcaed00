// The grouped MXFP4 product: row r of expert e is
//   y[r, n] = sum over blocks b of
//             2^(ea - 127) 2^(ew - 127) sum_j A[row(r), 32b + j] W[e, n, 32b + j],
// which v_mfma_scale_f32_32x32x64_f8f6f4 computes whole: e2m1 codes and the blocks' scale bytes go
// in as they lie in memory, sums stay in fp32.
//
// Operands: the weights are the MFMA's A (its rows are output columns n), the activations its B
// (its columns are routed rows), so a lane's 16 results are 4 runs of 4 consecutive n of one routed
// row.  Lane l of an operand holds one block of one row: row l % 32 and, of the MFMA's two blocks,
// l / 32, as 16 bytes of codes and one scale byte (a byte of a register that the instruction
// picks).  The order in which blocks are taken is free as long as both operands agree, so a lane
// takes runs of consecutive blocks.
#include <algorithm>
#include <type_traits>

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

// The expert whose tile `id` is, and the tile's rows.  Tiles of BM = 32 rows are numbered without a
// pass over the experts' counts: expert e's start at offsets[e] / BM + e, which leaves room for all
// of them (ceil(n / BM) <= (offsets[e] + n) / BM - offsets[e] / BM + 1) and grows by one at least
// from expert to expert, so a tile's expert is the last one whose first number is not above it.
// Some numbers belong to no tile: those workgroups end.  With fewer rows than that gives numbers, a
// tile is numbered by its first row instead (`by_row`).  The lanes compare 64 experts at a time, up
// to 512 experts' loads in flight together.
struct Tile {
  int expert, row0, nrows;
};
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ offsets, int E, int rows,
                                          int id, bool by_row) {
  constexpr int BM = 32;
  const int lane = threadIdx.x & 63;
  int upto = 0;  // experts whose first number is not above id: a prefix of them
  for (int e0 = 0; e0 < E; e0 += 512) {
    int o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      o[j] = e0 + 64 * j < E ? offsets[min(e0 + 64 * j + lane, E - 1)] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + 64 * j + lane;
      upto += __popcll(ballot(e < E && (by_row ? o[j] : o[j] / BM + e) <= id));
    }
  }
  Tile t;
  t.expert = max(upto - 1, 0);
  const int first = offsets[t.expert];
  const int last = min(offsets[t.expert + 1], rows);
  if (by_row) {
    t.row0 = id < first || (id - first) % BM != 0 ? last : id;
  } else {
    t.row0 = first + (id - (first / BM + t.expert)) * BM;
  }
  t.nrows = min(last - t.row0, BM);  // <= 0: no tile
  return t;
}

// silu(g) * u in fp32 with the hardware's exponential and reciprocal, 1 ulp each; the roundings of
// the exponent's argument and of its constant add 1.25 |g| 2^-24.  The result goes into 4 bits.
// From g = -87.4 down 1 + e is 2^126 or more, whose reciprocal the hardware takes for 0: the result
// is -0 where silu(g) is less than 2^-119 in magnitude.
__device__ __forceinline__ float swiglu(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896341f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// ---- few rows ------------------------------------------------------------------------------
// One workgroup: up to 32 rows of an expert by 32 columns (SwiGLU: 32 gates and their 32 ups), K
// split over its 4 wavefronts and joined in LDS.  With so few rows a call is bound by latency: each
// wavefront loads its operands from memory straight into the MFMA's layout, with no stage or
// barrier before the join.  One token's ten rows, gate/up (11 MB of weights): 7.0 us; down: 4.6 us.
template <int EPI>
__global__ __launch_bounds__(256) void mx_mm_narrow_kernel(MxProblem p, bool by_row) {
  constexpr int kMats = EPI == kMxSwiglu ? 2 : 1;
  __shared__ float part[4][kMats][32][36];
  const Tile t = find_tile(p.offsets, p.E, p.rows, blockIdx.x, by_row);
  if (t.nrows <= 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int n0 = blockIdx.y * 32;
  const size_t kb = p.k_in / 2, sb = p.k_in / kMxBlock;
  int r = t.row0 + min(l32, t.nrows - 1);
  r = p.src ? route_row(p.src[r], p.by_k.mul, p.by_k.shift, p.n_act) : min(r, p.n_act - 1);
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

  // 128 values at a time, up to kBatch times' loads under way before the first products
  constexpr int kBatch = 4;
  const int chunks = p.k_in / 128;
  for (int c0 = wave; c0 < chunks; c0 += 4 * kBatch) {
    v4i av[kBatch][2], wv[kBatch][kMats][2];
    int sa[kBatch], sw[kBatch][kMats];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int c = c0 + 4 * b;
      if (c >= chunks) break;  // uniform
      const v4i* ap = reinterpret_cast<const v4i*>(a + c * 64);
      av[b][0] = ap[0];
      av[b][1] = ap[1];
      sa[b] = *reinterpret_cast<const uint16_t*>(as + c * 4);
#pragma unroll
      for (int m = 0; m < kMats; ++m) {
        const v4i* wp = reinterpret_cast<const v4i*>(w + m * up * kb + c * 64);
        wv[b][m][0] = wp[0];
        wv[b][m][1] = wp[1];
        sw[b][m] = *reinterpret_cast<const uint16_t*>(ws + m * up * sb + c * 4);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (c0 + 4 * b >= chunks) break;
#pragma unroll
      for (int m = 0; m < kMats; ++m) {
        acc[m] = mfma_mx<0>(wv[b][m][0], av[b][0], acc[m], sw[b][m], sa[b]);
        acc[m] = mfma_mx<1>(wv[b][m][1], av[b][1], acc[m], sw[b][m], sa[b]);
      }
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
    float h[8], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = swiglu(y[0][j], y[1][j]);
      h[j + 4] = 0.0f;
      m = mx_amax(m, h[j]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = mx_amax(m, __shfl_xor(m, o));
    const uint32_t byte = mx_scale_byte(m);
    const uint32_t codes = mx_codes8(h, byte);
    if (live) {
      uint8_t* o = static_cast<uint8_t*>(p.out) + row * (p.n_out / 2) + (n0 + tc) / 2;
      *reinterpret_cast<uint16_t*>(o) = (uint16_t)codes;
      if ((threadIdx.x & 7) == 0)
        p.out_scales[row * (p.n_out / kMxBlock) + n0 / kMxBlock] = (uint8_t)byte;
    }
  } else if (live) {
    if constexpr (EPI == kMxF32) {
      float* o = static_cast<float*>(p.out) + row * p.n_out + n0 + tc;
      *reinterpret_cast<float4*>(o) = make_float4(y[0][0], y[0][1], y[0][2], y[0][3]);
    } else {
      typedef __bf16 v4 __attribute__((ext_vector_type(4)));
      __bf16* o = static_cast<__bf16*>(p.out) + row * p.n_out + n0 + tc;
      *reinterpret_cast<v4*>(o) =
          (v4){(__bf16)y[0][0], (__bf16)y[0][1], (__bf16)y[0][2], (__bf16)y[0][3]};
    }
  }
}

// ---- many rows -----------------------------------------------------------------------------
typedef __attribute__((address_space(3))) const void* lds_ptr_t;

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(lds_ptr_t)p;
}
// Direct global->LDS loads: lane i's 16 (4) bytes land at lds + 16 i (4 i), lds wave-uniform (M0);
// a lane's source is a uniform base and an offset of its own.  As inline assembly, so that the
// compiler does not wait for them at every LDS read (it cannot tell the buffers apart): the kernel
// waits for them itself. Nor does it then keep the distance between a vector instruction that
// writes a scalar register (a readlane, as it restores spilled scalars) and a load that takes its
// address from it, 5 wait states: the s_nop does, and covers the one that M0 needs.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
               : : "{m0}"(lds), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void dma4(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %1, %2"
               : : "{m0}"(lds), "v"(off), "s"(base) : "memory");
}

// A workgroup's tile: BN weight rows by BM routed rows, its wavefronts in WN slices of the columns
// by WM of the rows, each wavefront TN x TM MFMA tiles; row tiles are dealt to the WM in turn, so
// that few rows still keep all busy.  A stage is 256 values of K, 128 bytes of each row, in one of
// NBUF buffers.
constexpr int kStage = 128;
template <int WN_, int WM_, int TN_, int TM_, int NBUF_, int MINW_>
struct Geo {
  static constexpr int WN = WN_, WM = WM_, TN = TN_, TM = TM_, NBUF = NBUF_;
  static constexpr int kMinWaves = MINW_;  // wavefronts to fit on a SIMD
  static constexpr int kWaves = WN * WM;
  static constexpr int BN = WN * TN * 32, BM = WM * TM * 32, kRows = BN + BM;
  // loads of 16 bytes a lane: a stage's weight and routed rows (8 rows each), the scale bytes of
  // 512 values (64 rows each); or scale bytes of a stage, 4 bytes a lane (32 rows each).  A
  // wavefront issues every kWaves-th; where they do not come out even, the last is issued more than
  // once.
  static constexpr int kW = BN / 8, kA = BM / 8, kS = kRows / 64, kS4 = kRows / 32;
  static constexpr int kWI = (kW + kWaves - 1) / kWaves, kAI = (kA + kWaves - 1) / kWaves;
  static constexpr int kSI = (kS + kWaves - 1) / kWaves, kS4I = (kS4 + kWaves - 1) / kWaves;
  static constexpr int kBuf = kRows * kStage;
  static constexpr int kPerCu = MINW_ * 4 / kWaves;  // workgroups of a CU
  static_assert(BN % 64 == 0 && BM % 64 == 0 && kWaves * 4096 <= kBuf, "layout");
};
template <class G>
struct Lds {
  // a stage's weight rows, then its routed rows
  alignas(16) uint8_t rows[G::NBUF][G::kBuf];
  // their scale bytes: of 512 values, or of a stage
  alignas(16) uint8_t scales[G::NBUF][G::kRows * 16];
};

// Where a row's 16-byte piece c lies among its 8 in LDS: at c ^ swizzle(row).  Lanes of consecutive
// rows then read one piece index from different banks, in groups of 8 as of 16 lanes.
__device__ __forceinline__ int swizzle(int row) {
  return ((row >> 1) & 3) | (((row ^ (row >> 3)) & 1) << 2);
}

// Waits for the wavefront's loads to LDS, and for its LDS reads: what it read may be overwritten
// after the barrier.
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
}

// A wavefront's loads: uniform bases and its lanes' offsets.  WIDE: scale bytes come 16 of a row at
// a time (512 values), which K and the scales' alignment have to allow; otherwise 4 at a time, in
// every stage.
template <class G, bool WIDE>
struct Dma {
  static constexpr int kScales = WIDE ? G::kSI : G::kS4I;
  const uint8_t *w, *ws, *a, *as;
  uint32_t wo[G::kWI], ao[G::kAI], so[kScales];
  __device__ static int s_load(int i, int wave) {
    return WIDE ? min(wave + G::kWaves * i, G::kS - 1) : min(wave + G::kWaves * i, G::kS4 - 1);
  }
  __device__ static bool s_is_w(int i, int wave) {  // whether scale load i is of weight rows
    return WIDE ? s_load(i, wave) < G::BN / 64 : s_load(i, wave) < G::BN / 32;
  }
  // the tile row of a lane in scale load i, and its byte there
  __device__ static int s_row(int i, int wave, int lane) {
    return WIDE ? 64 * s_load(i, wave) + lane : 32 * s_load(i, wave) + lane / 2;
  }
  __device__ static int s_byte(int lane) { return WIDE ? 0 : 4 * (lane & 1); }
};

template <class G, bool WIDE, class WR>
__device__ __forceinline__ void plan_weights(Dma<G, WIDE>& d, int k_in, WR wrow, int wave,
                                             int lane) {
  const uint32_t kb = k_in / 2, sb = k_in / kMxBlock;
#pragma unroll
  for (int i = 0; i < G::kWI; ++i) {
    const int row = 8 * min(wave + G::kWaves * i, G::kW - 1) + lane / 8;
    d.wo[i] = wrow(row) * kb + 16 * ((lane & 7) ^ swizzle(row));
  }
#pragma unroll
  for (int i = 0; i < d.kScales; ++i) {
    const int row = d.s_row(i, wave, lane);
    if (row < G::BN) d.so[i] = wrow(row) * sb + d.s_byte(lane);
  }
}
// The routed rows' offsets, from the activation rows that arow(i) names.  FIRST: only the loads
// that arow makes, their results left in ao and so; otherwise the offsets from those.
template <class G, bool WIDE, bool FIRST, class AR>
__device__ __forceinline__ void plan_rows(Dma<G, WIDE>& d, int k_in, AR arow, int wave, int lane) {
  const uint32_t kb = k_in / 2, sb = k_in / kMxBlock;
#pragma unroll
  for (int i = 0; i < G::kAI; ++i) {
    const int row = 8 * min(wave + G::kWaves * i, G::kA - 1) + lane / 8;
    d.ao[i] = FIRST ? arow(row) : arow(d.ao[i]) * kb + 16 * ((lane & 7) ^ swizzle(row));
  }
#pragma unroll
  for (int i = 0; i < d.kScales; ++i) {
    const int row = d.s_row(i, wave, lane);
    if (row >= G::BN) d.so[i] = FIRST ? arow(row - G::BN) : arow(d.so[i]) * sb + d.s_byte(lane);
  }
}

// Load i of a stage's rows to LDS at `rows`, weight rows first; a stage's scale bytes to `scales`.
// `last_half`: of a last stage of 128 values, whose pieces 4..7 (scale bytes 4..7) do not exist;
// those lanes load the first ones again, and the products leave them out.
template <class G, bool WIDE>
__device__ __forceinline__ void issue_row(const Dma<G, WIDE>& d, int i, int stage, uint32_t rows,
                                          bool last_half, int wave, int lane) {
  const size_t k = (size_t)stage * kStage;
  auto off = [&](uint32_t o, int row) {
    if (WIDE || !last_half) return o;
    return o - ((((lane & 7) ^ swizzle(row)) & 4) ? 64u : 0u);
  };
  if (i < G::kWI) {
    const int l = min(wave + G::kWaves * i, G::kW - 1);
    dma16(d.w + k, off(d.wo[i], 8 * l + lane / 8), rows + 1024 * l);
  } else {
    const int j = i - G::kWI, l = min(wave + G::kWaves * j, G::kA - 1);
    dma16(d.a + k, off(d.ao[j], 8 * l + lane / 8), rows + G::BN * kStage + 1024 * l);
  }
}
template <class G, bool WIDE>
__device__ __forceinline__ void issue_scales(const Dma<G, WIDE>& d, int stage, uint32_t scales,
                                             bool last_half, int wave, int lane) {
  const size_t k = (size_t)stage * 8;
#pragma unroll
  for (int i = 0; i < d.kScales; ++i) {
    const uint8_t* base = (d.s_is_w(i, wave) ? d.ws : d.as) + k;
    if (WIDE)
      dma16(base, d.so[i], scales + 1024 * d.s_load(i, wave));
    else
      dma4(base, d.so[i] - (last_half ? d.s_byte(lane) : 0), scales + 256 * d.s_load(i, wave));
  }
}

// Where a lane reads in LDS: its piece of each of a stage's 4 steps in its wavefront's first weight
// and routed row tile, and its scale bytes.
struct Reads {
  const uint8_t *w[4], *a[4], *sw, *sa;
};
template <class G, bool WIDE>
__device__ __forceinline__ Reads plan_reads(const Lds<G>& lds, int wn, int wm, int lane) {
  const int l32 = lane & 31, half = lane >> 5, sz = swizzle(l32);  // tiles start at multiples of 32
  constexpr int kStride = WIDE ? 16 : 8;
  Reads r;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int at = l32 * kStage + 16 * ((4 * half + s) ^ sz);
    r.w[s] = lds.rows[0] + wn * G::TN * 32 * kStage + at;
    r.a[s] = lds.rows[0] + (G::BN + wm * 32) * kStage + at;
  }
  r.sw = lds.scales[0] + (wn * G::TN * 32 + l32) * kStride + 4 * half;
  r.sa = lds.scales[0] + (G::BN + wm * 32 + l32) * kStride + 4 * half;
  return r;
}

// The wavefront's products of one stage, with NL of its TM row tiles holding rows.  rows_at: the
// stage's buffer; scales_at: its set of scale bytes and place among its row's.  A wavefront that
// issues a load to LDS waits until the CU has taken it, about 200 clocks while all issue (a fifth
// to a half of a stage's time if it issues them in a row), so load(i), i < LOADS, are spread over
// the products, which go on meanwhile.
template <class G, bool WIDE, int NL, int LOADS, class F>
__device__ __forceinline__ void products(const Reads& r, int rows_at, int scales_at,
                                         v16f (&acc)[G::TN][G::TM], bool last_half, int lane,
                                         F load) {
  constexpr int kStride = WIDE ? 16 : 8;
  constexpr int N = NL > 0 ? NL : 1;
  // this lane's blocks do not exist: codes 0 at scale 1
  const bool none = !WIDE && last_half && lane >= 32;
  if constexpr (NL == 0) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load(i);
    return;
  }
  int sw[G::TN], sa[N];
#pragma unroll
  for (int j = 0; j < G::TN; ++j) {
    sw[j] = *reinterpret_cast<const int*>(r.sw + scales_at + j * 32 * kStride);
    if (!WIDE) sw[j] = none ? 0x7f7f7f7f : sw[j];
  }
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    sa[i] = *reinterpret_cast<const int*>(r.sa + scales_at + i * G::WM * 32 * kStride);
    if (!WIDE) sa[i] = none ? 0x7f7f7f7f : sa[i];
  }
  struct Operands {
    v4i w[G::TN], a[N];
  };
  auto read = [&](int s) {
    Operands o;
#pragma unroll
    for (int j = 0; j < G::TN; ++j) {
      o.w[j] = *reinterpret_cast<const v4i*>(r.w[s] + rows_at + j * 32 * kStage);
      if (!WIDE)
#pragma unroll
        for (int q = 0; q < 4; ++q) o.w[j][q] = none ? 0 : o.w[j][q];
    }
#pragma unroll
    for (int i = 0; i < NL; ++i)
      o.a[i] = *reinterpret_cast<const v4i*>(r.a[s] + rows_at + i * G::WM * 32 * kStage);
    return o;
  };
  constexpr int kSpread = 2 * N * G::TN;  // the first half of them: they land by the next stage
  Operands now = read(0);
  auto step = [&](auto S) {
    constexpr int s = decltype(S)::value;
    Operands next = now;
    if (s < 3) next = read(s + 1);
#pragma unroll
    for (int i = 0; i < NL; ++i)
#pragma unroll
      for (int j = 0; j < G::TN; ++j) {
        acc[j][i] = mfma_mx<s>(now.w[j], now.a[i], acc[j][i], sw[j], sa[i]);
        const int m = (s * NL + i) * G::TN + j;
        if (LOADS > 0 && m <= kSpread) {
#pragma unroll
          for (int l = m * LOADS / kSpread; l < LOADS && l < (m + 1) * LOADS / kSpread; ++l)
            load(l);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    now = next;
  };
  step(std::integral_constant<int, 0>{});
  step(std::integral_constant<int, 1>{});
  step(std::integral_constant<int, 2>{});
  step(std::integral_constant<int, 3>{});
}

// A copy that the compiler takes for a new value: what is computed from it stays where it is
// written instead of being kept in registers through the loops around it.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The wavefront's results for one row tile (32 rows from row0, `live` of them real) to memory.
// fp32 and bf16 tiles are turned in 4 KiB of LDS, so that 8 lanes write 128 bytes of a row.
template <class G, int EPI>
__device__ __forceinline__ void store_tile(const MxProblem& p, const v16f (&acc)[G::TN][G::TM],
                                           int i, size_t row0, int live, int n0, uint8_t* turn,
                                           int lane) {
  const int l32 = lane & 31, half = lane >> 5;
  if constexpr (EPI == kMxSwiglu) {
#pragma unroll
    for (int j = 0; j < G::TN / 2; ++j) {
      const int n = n0 + j * 32;
      if (n >= p.n_out) break;
      float lo[8], hi[8], m = 0.0f;  // columns 8g + 4 half + 0..3, for g = 0, 1 and 2, 3
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        lo[q] = swiglu(acc[j][i][q], acc[j + G::TN / 2][i][q]);
        hi[q] = swiglu(acc[j][i][q + 8], acc[j + G::TN / 2][i][q + 8]);
        m = mx_amax(mx_amax(m, lo[q]), hi[q]);
      }
      m = mx_amax(m, __shfl_xor(m, 32));
      const uint32_t byte = mx_scale_byte(m);
      const uint32_t c0 = mx_codes8(lo, byte), c1 = mx_codes8(hi, byte);  // 16 bits for each g
      const uint32_t o0 = (uint32_t)__shfl_xor((int)c0, 32), o1 = (uint32_t)__shfl_xor((int)c1, 32);
      if (l32 < live && half == 0) {
        const size_t row = row0 + l32;
        uint8_t* o = static_cast<uint8_t*>(p.out) + row * (p.n_out / 2) + n / 2;
        *reinterpret_cast<uint4*>(o) =
            make_uint4((c0 & 0xffffu) | (o0 << 16), (c0 >> 16) | (o0 & 0xffff0000u),
                       (c1 & 0xffffu) | (o1 << 16), (c1 >> 16) | (o1 & 0xffff0000u));
        p.out_scales[row * (p.n_out / kMxBlock) + n / kMxBlock] = (uint8_t)byte;
      }
    }
  } else {
    typedef __bf16 v4b __attribute__((ext_vector_type(4)));
    constexpr int kSize = EPI == kMxF32 ? 4 : 2;
    constexpr int kTiles = EPI == kMxF32 ? 1 : 2;  // column tiles of 128 bytes
    static_assert(G::TN % kTiles == 0, "whole 128-byte rows");
#pragma unroll
    for (int j0 = 0; j0 < G::TN; j0 += kTiles) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        const v16f& y = acc[j0 + j][i];
#pragma unroll
        for (int g = 0; g < 4; ++g) {  // columns 32 j + 8 g + 4 half + 0..3
          const int byte = (32 * j + 8 * g + 4 * half) * kSize;
          uint8_t* o = turn + l32 * 128 + 16 * ((byte / 16) ^ (l32 & 7)) + byte % 16;
          if constexpr (EPI == kMxF32)
            *reinterpret_cast<float4*>(o) =
                make_float4(y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]);
          else
            *reinterpret_cast<v4b*>(o) =
                (v4b){(__bf16)y[4 * g], (__bf16)y[4 * g + 1], (__bf16)y[4 * g + 2],
                      (__bf16)y[4 * g + 3]};
        }
      }
      const int n = n0 + j0 * 32 + (lane & 7) * (16 / kSize);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 8 * k + lane / 8;
        const uint4 v =
            *reinterpret_cast<const uint4*>(turn + r * 128 + 16 * ((lane & 7) ^ (r & 7)));
        if (r < live && n < p.n_out)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                    ((row0 + r) * p.n_out + n) * kSize) = v;
      }
    }
  }
}

// Where the workgroup is in its buffers: the one at work, and the sets of scale bytes at work and
// last loaded.
struct Ring {
  int buf = 0, set = -1, loaded = -1;
};

template <class G, bool WIDE>
__device__ __forceinline__ void issue_stage_scales(const Dma<G, WIDE>& d, int k, bool last_half,
                                                   Ring& ring, uint32_t lscales, int wave,
                                                   int lane) {
  if (WIDE && (k & 1) != 0) return;
  ring.loaded = (ring.loaded + 1) & (G::NBUF - 1);
  issue_scales(d, k, lscales + ring.loaded * G::kRows * 16, last_half, wave, lane);
}

// The tile's products along K.  `between` is called once a stage.  With two buffers each stage's
// loads are issued among the products of the one before it: its first stage's were before this, and
// its last stage issues the first of the next tile, which `turn_over` puts in place of this one in
// d.
template <class G, bool WIDE, int NL, class F, class A>
__device__ __forceinline__ void main_loop(const Reads& r, Dma<G, WIDE>& d, Ring& ring,
                                          uint32_t lrows, uint32_t lscales,
                                          v16f (&acc)[G::TN][G::TM], int k_in, F between,
                                          A turn_over, int wave, int lane) {
  constexpr int kLoads = G::kWI + G::kAI;
  const int stages = (k_in + 255) / 256;
  auto half_stage = [&](int k) { return !WIDE && 256 * (k + 1) > k_in; };
  for (int k = 0; k < stages; ++k) {
    wait_and_barrier();
    if constexpr (G::NBUF == 1) {
      issue_stage_scales(d, k, half_stage(k), ring, lscales, wave, lane);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) issue_row(d, i, k, lrows, half_stage(k), wave, lane);
      between();
      wait_and_barrier();
    }
    if (!WIDE || (k & 1) == 0) ring.set = (ring.set + 1) & (G::NBUF - 1);
    const int scales_at = ring.set * G::kRows * 16 + (WIDE ? (k & 1) * 8 : 0);
    if constexpr (G::NBUF == 2) {
      // after the products while other wavefronts' still go on; the largest tile has no registers
      // for that
      constexpr bool kAfter = G::TM <= 2;
      if (!kAfter) between();
      const int kn = k + 1 < stages ? k + 1 : 0;
      if (kn == 0) turn_over();
      issue_stage_scales(d, kn, half_stage(kn), ring, lscales, wave, lane);
      products<G, WIDE, NL, kLoads>(
          r, ring.buf * G::kBuf, scales_at, acc, half_stage(k), lane, [&](int i) {
            issue_row(d, i, kn, lrows + (ring.buf ^ 1) * G::kBuf, half_stage(kn), wave, lane);
          });
      if (kAfter) between();
      if (k + 1 < stages) ring.buf ^= 1;
    } else {
      products<G, WIDE, NL, 0>(r, 0, scales_at, acc, half_stage(k), lane, [](int) {});
    }
  }
}

// The lane's sum of v over the lanes up to it: within rows of 16 lanes, then over the rows.
__device__ __forceinline__ int scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Workgroups that stay: kPerCu of them on each CU, each with a share of the (row tile, column tile)
// pairs of all experts, and the next pair's place found and its rows' offsets computed while the
// products of the one at work go on.  (With a workgroup to a pair those two took 5.8 of its 20.6 us
// at 8192 tokens, 512 experts, gate/up.)
template <class G, int EPI, bool WIDE>
__global__ __launch_bounds__(G::kWaves * 64, G::kMinWaves) void mx_mm_wide_kernel(
    MxProblem p, uint32_t n_tiles) {
  __shared__ Lds<G> lds;
  constexpr bool kSwiglu = EPI == kMxSwiglu;
  constexpr int kFeat = kSwiglu ? G::BN / 2 : G::BN;  // output columns of a tile
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % G::WN, wm = wave / G::WN;

  // Lane l counts the row tiles of experts l * seg .. l * seg + seg - 1, and of all before them.
  const int seg = (p.E + 63) / 64;
  auto tiles_of = [](int n) { return (max(n, 0) + G::BM - 1) / G::BM; };
  int before = 0, prev = min(p.offsets[min(lane * seg, p.E)], p.rows);
  for (int i = 1; i <= seg; ++i) {
    const int o = min(p.offsets[min(lane * seg + i, p.E)], p.rows);
    before += tiles_of(o - prev);
    prev = o;
  }
  const int upto = scan(before);
  const uint32_t pairs = (uint32_t)__builtin_amdgcn_readlane(upto, 63) * n_tiles;
  before = upto - before;

  // Workgroups go to the 8 XCDs in turn.  Each XCD takes an eighth of the pairs, column tiles
  // fastest, and its workgroups walk through it side by side: at any time they share a few experts'
  // weights and rows in the XCD's L2.
  const uint32_t xcd = blockIdx.x & 7, step = gridDim.x >> 3;
  const uint32_t end = (uint32_t)((uint64_t)pairs * (xcd + 1) >> 3);
  uint32_t pair = (uint32_t)((uint64_t)pairs * xcd >> 3) + (blockIdx.x >> 3);
  if (pair >= end) return;

  Dma<G, WIDE> d, e;  // the loads of the pair at work and of the next
  d.a = p.a;
  d.as = p.as;
  e = d;
  Tile t, u;
  int n0, un0, piece = 0;
  int at = 0;  // how far the next pair is
  // The next pair in three steps, each of which uses what the one before has loaded: its segment of
  // the offsets; its tile, and the activation rows; all offsets.
  auto advance = [&](uint32_t next) {
    if (at == 0) {
      const int q = (int)(next / n_tiles);
      un0 = (int)(next % n_tiles) * kFeat;
      const int s = __popcll(ballot(before <= q)) - 1;  // the last lane that is not past it
      u.row0 = q - __builtin_amdgcn_readlane(before, s);
      u.expert = s * seg;
      piece = p.offsets[min(u.expert + lane, p.E)];
      at = 1;
    } else if (at == 1) {
      const int o = min(piece, p.rows), n = max(__shfl_down(o, 1) - o, 0);
      const int mine = lane < seg && u.expert + lane < p.E ? tiles_of(n) : 0;
      const int incl = scan(mine);
      const int s = __popcll(ballot(incl <= u.row0));  // lanes all of whose tiles come before
      const int m = u.row0 -
                    (__builtin_amdgcn_readlane(incl, s) - __builtin_amdgcn_readlane(mine, s));
      const int rows = __builtin_amdgcn_readlane(n, s), count = __builtin_amdgcn_readlane(mine, s);
      // an expert's tiles are equally high, to 32 rows
      const int high = ((rows + count - 1) / count + 31) / 32 * 32;
      u.expert += s;
      u.row0 = __builtin_amdgcn_readlane(o, s) + m * high;
      u.nrows = min(rows - m * high, high);
      auto load = [&](int i) -> uint32_t {
        const int r = u.row0 + min(i, u.nrows - 1);
        return p.src ? p.src[r] : r;
      };
      plan_rows<G, WIDE, true>(e, p.k_in, load, wave, here(lane));
      at = 2;
    } else if (at == 2) {
      auto act = [&](uint32_t r) -> uint32_t {
        return p.src ? route_row((int32_t)r, p.by_k.mul, p.by_k.shift, p.n_act)
                     : min(r, (uint32_t)(p.n_act - 1));
      };
      plan_rows<G, WIDE, false>(e, p.k_in, act, wave, here(lane));
      auto wrow = [&](int i) -> uint32_t {  // the expert's matrix row in row i of the tile
        if constexpr (kSwiglu) {  // half of a wavefront's TN tiles are gates, then their ups
          const int tile = i >> 5, slice = tile / G::TN, j = tile % G::TN;
          const int f = un0 + (slice * (G::TN / 2) + j % (G::TN / 2)) * 32 + (i & 31);
          return min(f, p.n_out - 1) + (j >= G::TN / 2 ? p.n_out : 0);
        } else {
          return min(un0 + i, p.n_out - 1);
        }
      };
      const size_t mat = (size_t)u.expert * p.n_out * (kSwiglu ? 2 : 1);
      e.w = p.w + mat * (p.k_in / 2);
      e.ws = p.ws + mat * (p.k_in / kMxBlock);
      plan_weights(e, p.k_in, wrow, wave, here(lane));
      at = 3;
    }
  };

  uint32_t lrows = lds_address(lds.rows), lscales = lds_address(lds.scales);
  asm volatile("" : "+s"(lrows), "+s"(lscales));
  const Reads r = plan_reads<G, WIDE>(lds, wn, wm, lane);
  while (at < 3) advance(pair);
  Ring ring;
  d = e;
  if (G::NBUF == 2) {
    const bool last_half = !WIDE && p.k_in < 256;
    issue_stage_scales(d, 0, last_half, ring, lscales, wave, lane);
#pragma unroll
    for (int i = 0; i < G::kWI + G::kAI; ++i) issue_row(d, i, 0, lrows, last_half, wave, lane);
  }
  for (;;) {
    t = u, n0 = un0, at = 0;
    if (G::NBUF == 1) d = e;
    const uint32_t next = pair + step;
    auto between = [&]() {
      if (next < end) advance(next);
    };
    auto turn_over = [&]() {  // after the last pair its first stage is loaded again, for nothing
      if (next >= end) return;
      while (at < 3) advance(next);
      d = e;
    };
    const int row_tiles = (t.nrows + 31) / 32;
    const int live = row_tiles > wm ? (row_tiles - wm + G::WM - 1) / G::WM : 0;
    auto go = [&](auto N) {  // one instance for each number of row tiles
      constexpr int NL = decltype(N)::value;
      if constexpr (NL <= G::TM) {
        if (live != NL) return;
        v16f acc[G::TN][G::TM];
#pragma unroll
        for (int j = 0; j < G::TN; ++j)
#pragma unroll
          for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[j][i][q] = 0.0f;
        main_loop<G, WIDE, NL>(r, d, ring, lrows, lscales, acc, p.k_in, between, turn_over, wave,
                               lane);
        if (!kSwiglu) {  // tiles are turned in the stage's buffer once all are done with it
          asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" : : : "memory");
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int r0 = __builtin_amdgcn_readfirstlane(here((i * G::WM + wm) * 32));
          store_tile<G, EPI>(p, acc, i, (size_t)t.row0 + r0, min(t.nrows - r0, 32),
                             n0 + wn * (kFeat / G::WN), lds.rows[ring.buf] + 4096 * wave,
                             here(lane));
        }
      }
    };
    go(std::integral_constant<int, 0>{});
    go(std::integral_constant<int, 1>{});
    go(std::integral_constant<int, 2>{});
    go(std::integral_constant<int, 3>{});
    go(std::integral_constant<int, 4>{});
    static_assert(G::TM <= 4, "instances");
    if (next >= end) break;
    while (at < 3) advance(next);
    if (G::NBUF == 2) ring.buf ^= 1;
    pair = next;
  }
  if (G::NBUF == 2) wait_and_barrier();  // no load to LDS is under way when the workgroup ends
}

constexpr int kCus = 256;  // MI355X
template <class G, int EPI>
hipError_t launch_wide(const MxProblem& p, hipStream_t s) {
  const int feat = EPI == kMxSwiglu ? G::BN / 2 : G::BN;
  const uint32_t n_tiles = (p.n_out + feat - 1) / feat;
  const uint64_t most = (uint64_t)(p.rows / G::BM + (p.E < p.rows ? p.E : p.rows)) * n_tiles;
  unsigned grid = kCus * G::kPerCu;
  if (most < grid) grid = (unsigned)(most + 7) / 8 * 8;
  if (p.k_in % 512 == 0 && ((uintptr_t)p.ws | (uintptr_t)p.as) % 16 == 0)
    mx_mm_wide_kernel<G, EPI, true><<<grid, G::kWaves * 64, 0, s>>>(p, n_tiles);
  else
    mx_mm_wide_kernel<G, EPI, false><<<grid, G::kWaves * 64, 0, s>>>(p, n_tiles);
  return hipGetLastError();
}
hipError_t launch_narrow(const MxProblem& p, hipStream_t s) {
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
template <class G>
hipError_t launch_wide_any(const MxProblem& p, hipStream_t s) {
  return p.epilogue == kMxF32    ? launch_wide<G, kMxF32>(p, s)
         : p.epilogue == kMxBF16 ? launch_wide<G, kMxBF16>(p, s)
                                 : launch_wide<G, kMxSwiglu>(p, s);
}

}  // namespace

// Which kernel, by sizes alone (us, MI355X; columns: the narrow kernel, then the wide one's tiles,
// whose last two have two buffers):
//                                   narrow  256 x 64  128 x 192  256 x 256  128 x 128
//   gate/up 2048 -> 2 x 512, 512 experts, K = 10
//     1 token                          7.0      11.8                              9.3
//     4 tokens                        13.8      15.0                             14.3
//     16 tokens                       39.6      35.6       34.9       40.1       34.8
//     2048 tokens (40 rows each)       341       118        137        147        140
//     8192 tokens (160 rows)           903       204        179        180        239
//     32768 tokens (640 rows)         2994       644        578        480        597
//   down 512 -> 2048, 512 experts, K = 10
//     16 tokens                       23.1      19.4       22.5       26.0       24.4
//     8192 tokens                      600       160        144        166        207
//   one 4096 x 4096 matrix
//     16 rows                          9.6      20.4       19.2       19.5       14.3
//     256 rows                        33.2      24.5       23.3       31.3       17.5
//     1024 rows                         99      29.2       31.6       31.6       21.1
//     8191 rows                        707       112        112         88        112
// The narrow kernel wins while its workgroups all run at once, 3 to a CU; 128 x 128 while larger
// tiles would not fill the CUs twice; then the tile's height goes by the rows an expert has.
hipError_t launch_mx_mm(const MxProblem& p_, hipStream_t s) {
  MxProblem p = p_;
  p.by_k = division_by(p.K);
  auto tiles = [&](int high) { return std::min<int64_t>(p.rows, (int64_t)p.rows / high + p.E); };
  if (tiles(32) * (p.n_out / 32) <= 3 * kCus) return launch_narrow(p, s);
  const int64_t feat = p.epilogue == kMxSwiglu ? 128 : 256;
  if (tiles(128) * ((p.n_out + feat - 1) / feat) < 2 * kCus)
    return launch_wide_any<Geo<2, 2, 2, 2, 2, 2>>(p, s);
  const int mean = p.rows / p.E;
  if (mean <= 64) return launch_wide_any<Geo<4, 1, 2, 2, 1, 3>>(p, s);
  if (mean <= 192) return launch_wide_any<Geo<2, 2, 2, 3, 1, 3>>(p, s);
  return launch_wide_any<Geo<4, 2, 2, 4, 2, 2>>(p, s);
}

}  // namespace moe
