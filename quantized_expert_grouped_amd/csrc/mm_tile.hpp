// The grouped products' tile kernel: D[i, j] = sum_c P[i, c] Q[j, c] for a tile of BI x BJ results
// at a time, c in stages of 32 or 64.
//
// A stage of an operand goes from memory straight into one of two or four LDS buffers
// (buffer_load_dwordx4 ... lds).  An operand whose c is contiguous in memory (w and a in the
// forward, grad in dgrad) lies there as rows of a stage's c; one whose i or j is contiguous (w
// in dgrad, both in wgrad) as a stage's rows of BI or BJ values, and is turned by the LDS read itself
// (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 values, and each gets a column of 4).  Both are
// stored with their 16-byte pieces in an order that lets the lanes of a read take different banks.
// A piece that is not there (past the matrix's edge, the last row, the end of c) has an offset past
// the buffer descriptor's size, for which the load writes zeros without a fetch.
//
// What bounds it (us, MI355X): 8191 x 4096 x 4096 forward 226 to 243 (1130 to 1215 TFLOP/s; the matrix
// cores are busy for 61% of the cycles, LDS reads find no bank conflict), dgrad 224 to 243, wgrad 223
// to 250.  8192 tokens, K = 10, 512 experts, 2048 -> 2 x 512: memory in the forward, 2.4 GB in 547 to
// 590, and in dgrad, 2.65 GB in 577 to 591; wgrad, 2.35 GB (2.1 written) in 771 to 780, is bound by
// neither memory nor the matrix cores (3.0 TB/s; busy for 20% of the cycles): a tile is five or six stages
// and then 128 KB of results, and the one workgroup of a CU has nothing else to do while they drain.
//
// Workgroups stay and walk through the tiles.  Loads run as many stages ahead of the products as
// there are buffers, over the tiles' ends: a stage's go out into the buffer whose reads have just
// ended, while with four those of two others are still on their way.
#pragma once

#include "mm.hpp"

namespace moe {

namespace tile {

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) const void* lds_ptr_t;

constexpr uint32_t kNone = 0x80000000u;   // an offset with this bit is past the descriptors' size
__device__ __forceinline__ uint32_t none_if(bool none) { return none ? kNone : 0u; }

// Wavefronts: WI slices of i by WJ of j, each TI x TJ MFMA tiles of 32 x 32; j's tiles are dealt to
// the WJ in turn, so that few rows still keep all busy.  C c's make a stage, a step of the matrix
// instruction 16 of them; BUFS stages have buffers.
template <int WI_, int WJ_, int TI_, int TJ_, int C_, int BUFS_>
struct Geo {
  static constexpr int WI = WI_, WJ = WJ_, TI = TI_, TJ = TJ_, kC = C_, kBufs = BUFS_;
  static constexpr int kSteps = kC / 16;
  static constexpr int kWaves = WI * WJ, BI = WI * TI * 32, BJ = WJ * TJ * 32;
  static constexpr int kPL = BI * kC / 512 / kWaves, kQL = BJ * kC / 512 / kWaves;  // loads of 1 KB
  static constexpr int kBuf = (BI + BJ) * kC * 2;
  static constexpr int kPerCu = kBufs * kBuf > 65536 ? 1 : 2;  // workgroups of a CU
  static_assert(TI == 2 && BI * kC % (512 * kWaves) == 0 && BJ * kC % (512 * kWaves) == 0 &&
                    (kC == 32 || kC == 64) && kBufs >= 2,
                "whole loads");
  static_assert((BI & (BI - 1)) == 0 && (BJ & (BJ - 1)) == 0 && kBuf >= kWaves * 4096, "layout");
};

// OWN: the wavefronts have 4 KB each of their own to turn their results in; otherwise the experts'
// offsets are here, and results are turned in a stage's buffer.
template <class G, bool OWN>
struct Lds {
  alignas(1024) uint8_t buf[G::kBufs][G::kBuf];  // P's stage, then Q's
  alignas(16) uint8_t more[OWN ? G::kWaves * 4096 : (kMaxExperts + 1) * 4];
};

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(lds_ptr_t)p;
}

// Lane l's 16 bytes at base + off land at lds + 16 l.  As inline assembly, so that the compiler does
// not wait for it at every LDS read; the kernel waits itself.  The s_nop keeps the distance that a
// scalar register written by a vector instruction (a readlane) needs before a memory instruction
// reads it, and m0's.
__device__ __forceinline__ void dma16(uint64_t base, uint32_t off, uint32_t lds) {
  const v4i rsrc = {__builtin_amdgcn_readfirstlane((int)(uint32_t)base),
                    __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32)), (int)kNone,
                    0x00020000};
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               : : "{m0}"(lds), "v"(off), "s"(rsrc) : "memory");
}

// Waits for all but the last KEEP of the wavefront's accesses to memory, and for its LDS reads.
template <int KEEP = 0>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(KEEP) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
}
__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
}

// Between lanes of one wavefront, whose LDS operations complete in order, nothing has to wait; but
// the compiler is to keep what was written by other lanes apart from what was there before.
__device__ __forceinline__ void lanes_fence() {
  asm volatile("" : : : "memory");
  __builtin_amdgcn_wave_barrier();
}

// A copy that the compiler takes for a new value: what is computed from it stays where it is
// written instead of being kept in registers through the loops around it.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Where piece c of a narrow row lies among its 4 or 8: at c ^ swizzle(row).
template <int C>
__device__ __forceinline__ int swizzle(int row) {
  if (C == 32) return (row >> 2) & 3;
  return ((row >> 1) & 3) | (((row ^ (row >> 3)) & 1) << 2);
}

// Read by scalar loads, which no wait for vector ones holds up (nor do they wait for stores).
typedef __attribute__((address_space(4))) const int32_t* scalar_ptr_t;
__device__ __forceinline__ scalar_ptr_t constant(const int32_t* p) {
  return (scalar_ptr_t)(uintptr_t)p;
}

// A tile's place and its reduction.
struct Tile {
  int expert, row0, nrows, i0, j0, nc;
};

// One operand's stage of C c's, B indices wide.  kWide: c is not the contiguous index.
template <int B, int C, int kLoads, int kWaves, bool kWide>
struct Operand {
  uint64_t base;
  uint32_t off[kLoads];
  static constexpr int kRow = B * 2;             // bytes of a c row
  static constexpr int kRows = 1024 / kRow;      // of them in a load
  static constexpr int kLanes = 64 / kRows;      // lanes of each
  static_assert(!kWide || (B >= 128 && B <= 512), "rows of four 64-byte chunks, whole in a load");

  // Load l: this lane's index (narrow) or c (wide), and the first c or index of its piece.
  __device__ static int row(int l, int lane) {
    return kWide ? l * kRows + lane / kLanes : 512 / C * l + lane / (C / 8);
  }
  __device__ static int first(int l, int lane) {
    if (kWide) return ((lane % kLanes) ^ ((row(l, lane) & 3) << 2)) * 8;
    return (lane % (C / 8) ^ swizzle<C>(row(l, lane))) * 8;
  }
  __device__ __forceinline__ void issue(int i, uint32_t lds, int wave) const {
    const int l = wave + kWaves * i;
    dma16(base, off[i], lds + 1024 * l);
  }
  // The last stage has only `left` c's.
  __device__ __forceinline__ void mask(int left, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int l = wave + kWaves * i;
      off[i] |= none_if((kWide ? row(l, lane) : first(l, lane)) >= left);
    }
  }
};

// Where a lane reads an operand: TN tiles, kStep index tiles apart.
template <int B, int C, int TN, int kStep, bool kWide>
struct Reader {
  uint32_t at[kWide ? TN : C / 16];
  __device__ __forceinline__ void plan(uint32_t lds, int first_tile, int lane) {
    if constexpr (kWide) {
      const int l16 = lane & 15;
#pragma unroll
      for (int t = 0; t < TN; ++t)
        at[t] = lds + (8 * (lane >> 5) + (l16 >> 2)) * (B * 2) +
                (((first_tile + t * kStep) ^ (l16 >> 2)) * 64) + 32 * ((lane >> 4) & 1) +
                8 * (l16 & 3);
    } else {
      const int row = lane & 31;
#pragma unroll
      for (int s = 0; s < C / 16; ++s)
        at[s] = lds + (first_tile * 32 + row) * (C * 2) +
                16 * ((2 * s + (lane >> 5)) ^ swizzle<C>(row));
    }
  }
  // 16 c's of tile t in step s
  __device__ __forceinline__ v4i read(int t, int s, uint32_t buf) const {
    typedef __attribute__((address_space(3))) const v4i* pv4i;
    typedef __attribute__((address_space(3))) v4s* pv4s;
    if constexpr (kWide) {
      const uint32_t a = at[t] + buf + 16 * s * (B * 2);
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((pv4s)(uintptr_t)a);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((pv4s)(uintptr_t)(a + 4 * (B * 2)));
      const v2i l = __builtin_bit_cast(v2i, lo), h = __builtin_bit_cast(v2i, hi);
      return (v4i){l[0], l[1], h[0], h[1]};
    } else {
      return *(pv4i)(uintptr_t)(at[s] + buf + t * kStep * 32 * C * 2);
    }
  }
};

template <int OP, int DT, int ODT, bool SWIGLU, class G>
struct Kernel {
  static constexpr bool kGates = OP == kMmForward && SWIGLU;
  static constexpr bool kPWide = OP != kMmForward, kQWide = OP == kMmWgrad;
  static constexpr int kC = G::kC, kBufs = G::kBufs;
  typedef Operand<G::BI, kC, G::kPL, G::kWaves, kPWide> OpP;
  typedef Operand<G::BJ, kC, G::kQL, G::kWaves, kQWide> OpQ;
  // Tiles of j that are walked through together: the workgroups of an XCD, side by side, then share
  // what they read in a squarer patch (8191 x 4096 x 4096, 1 and 4: dgrad 246 and 243 us, wgrad 248
  // and 236).
  static constexpr uint32_t kGroup = 4;
  static constexpr int kFeat = kGates ? G::BI / 2 : G::BI;  // i's of a tile

  // wgrad's results need nothing but their rounding, and its tiles can be short: their ends must not
  // hold up the loads
  static constexpr bool kOwnTurn = OP == kMmWgrad;
  typedef Lds<G, kOwnTurn> L;

  const MmProblem& p;
  L& lds;
  int32_t* const offsets;
  const int lane, wave, wi, wj;
  uint32_t ni_tiles, nj_tiles;  // i's tiles, and of all experts j's
  uint32_t per_expert;          // wgrad: of one expert
  int before, seg;  // fwd, dgrad: row tiles of the experts before this lane's segment of seg

  __device__ Kernel(const MmProblem& p_, L& l)
      : p(p_), lds(l), offsets(reinterpret_cast<int32_t*>(l.more)), lane(threadIdx.x & 63),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), wi(wave % G::WI),
        wj(wave / G::WI) {}

  __device__ __forceinline__ int ni() const { return OP == kMmForward ? p.n_out : p.k_in; }

  // The tiles there are, in pairs (or, wgrad, triples) of which i's tile is the fastest.
  __device__ __forceinline__ uint32_t count() {
    ni_tiles = (uint32_t)(ni() + kFeat - 1) / kFeat;
    if constexpr (OP == kMmWgrad) {
      per_expert = (uint32_t)(p.n_out + G::BJ - 1) / G::BJ;
      nj_tiles = (uint32_t)p.E * (uint32_t)p.parts * per_expert;
      return nj_tiles * ni_tiles;
    } else {
      for (int e = threadIdx.x; e <= p.E; e += G::kWaves * 64)
        offsets[e] = min(p.offsets[e], p.rows);
      __syncthreads();
      seg = (p.E + 63) / 64;
      int mine = 0;
      for (int i = 0; i < seg; ++i) {
        const int e = lane * seg + i;
        if (e < p.E) mine += tiles_of(offsets[e + 1] - offsets[e]);
      }
      before = lane_scan(mine);
      nj_tiles = (uint32_t)__builtin_amdgcn_readlane(before, 63);
      before -= mine;
      return nj_tiles * ni_tiles;
    }
  }
  __device__ static int tiles_of(int n) { return (max(n, 0) + G::BJ - 1) / G::BJ; }

  __device__ __forceinline__ Tile find(uint32_t q) const {
    Tile t;
    // kGroup tiles of j to all of i's, then the next
    const uint32_t g = q / (ni_tiles * kGroup), in = q - g * (ni_tiles * kGroup);
    const uint32_t high = min(kGroup, nj_tiles - g * kGroup);
    const int qi = (int)(in / high);
    int qr = (int)(g * kGroup + in - qi * high);
    t.i0 = qi * kFeat;
    if constexpr (OP == kMmWgrad) {
      t.expert = qr / (int)per_expert;  // of p.parts to an expert, each with a part of its rows
      t.j0 = (qr - t.expert * (int)per_expert) * G::BJ;
      const int e = p.parts > 1 ? t.expert / p.parts : t.expert;
      t.row0 = min(constant(p.offsets)[e], p.rows);
      t.nc = max(min(constant(p.offsets)[e + 1], p.rows) - t.row0, 0);
      if (p.parts > 1) {
        const int part = ((t.nc + p.parts - 1) / p.parts + kC - 1) / kC * kC;
        const int at = min((t.expert - e * p.parts) * part, t.nc);
        t.row0 += at;
        t.nc = min(t.nc - at, part);
      }
      t.nrows = min(p.n_out - t.j0, G::BJ);
    } else {
      const int s = __popcll(ballot(before <= qr)) - 1;  // the last segment that is not past it
      const int e = s * seg + lane;
      const bool on = lane < seg && e < p.E;
      const int o = on ? offsets[e] : 0, n = on ? offsets[e + 1] - o : 0;
      const int mine = on ? tiles_of(n) : 0, incl = lane_scan(mine);
      qr -= __builtin_amdgcn_readlane(before, s);
      const int x = __popcll(ballot(incl <= qr));  // lanes all of whose tiles come before
      const int m = qr - (__builtin_amdgcn_readlane(incl, x) - __builtin_amdgcn_readlane(mine, x));
      const int rows = __builtin_amdgcn_readlane(n, x), many = __builtin_amdgcn_readlane(mine, x);
      const int high = ((rows + many - 1) / many + 31) / 32 * 32;  // equally high, to 32 rows
      t.expert = s * seg + x;
      t.row0 = __builtin_amdgcn_readlane(o, x) + m * high;
      t.nrows = min(rows - m * high, high);
      t.j0 = 0;
      t.nc = OP == kMmForward ? p.k_in : p.n_out;
    }
    return t;
  }

  // ---- loads ----
  struct Loads {
    OpP P;
    OpQ Q;
    int left;             // c's from the next stage on
    int row;              // wgrad with src: the next stage's first row,
    uint32_t at;          //   and where in a row of a this lane's pieces lie
    // forward: each lane's row's; wgrad: those of each load's rows, the same in all lanes
    int route[OP == kMmWgrad ? G::kPL * OpP::kRows : OP == kMmForward ? G::kQL : 1];
  };

  // The routes that the next stage's loads need, fetched a stage ahead: of the tile's next rows, or
  // of the next tile's first.
  __device__ __forceinline__ void fetch(Loads& d, const Tile& t, int row0, int left) const {
    if (OP == kMmDgrad || !p.src) return;
    const int lane = here(this->lane);
    if constexpr (OP == kMmForward) {
#pragma unroll
      for (int i = 0; i < G::kQL; ++i)
        d.route[i] = p.src[t.row0 + min(OpQ::row(wave + G::kWaves * i, lane), t.nrows - 1)];
    } else {
#pragma unroll
      for (int i = 0; i < G::kPL; ++i)
#pragma unroll
        for (int h = 0; h < OpP::kRows; ++h) {
          const int c = (wave + G::kWaves * i) * OpP::kRows + h;
          // (a row past the last is not fetched; its route is one that is there)
          d.route[i * OpP::kRows + h] =
              constant(p.src)[min(row0 + min(c, max(left - 1, 0)), p.rows - 1)];
        }
    }
  }

  __device__ __forceinline__ void plan(Loads& d, const Tile& t) const {
    constexpr int kSize = 2;
    const int lane = here(this->lane);
    const uint64_t w = (uint64_t)p.w + (uint64_t)t.expert * (kGates ? 2 : 1) * p.n_out * p.k_in * kSize;
    const uint64_t a = (uint64_t)p.a, g = (uint64_t)p.grad;
    d.left = t.nc;
    if constexpr (OP == kMmForward) {
      d.P.base = w;
#pragma unroll
      for (int i = 0; i < G::kPL; ++i) {
        const int l = wave + G::kWaves * i, x = OpP::row(l, lane);
        int f = t.i0 + x, n = f;
        if constexpr (kGates) {  // a wavefront's two tiles are gates and their ups
          f = t.i0 + (x >> 6) * 32 + (x & 31);
          n = f + (x & 32 ? p.n_out : 0);
        }
        d.P.off[i] =
            ((uint32_t)n * (uint32_t)p.k_in + OpP::first(l, lane)) * kSize | none_if(f >= p.n_out);
      }
    } else {
      const int64_t ld = OP == kMmDgrad ? p.k_in : p.lda;
      const bool gathered = OP == kMmWgrad && p.src;
      d.P.base = OP == kMmDgrad ? w : gathered ? a : a + (uint64_t)(t.row0 * ld * kSize);
      const int x = t.i0 + OpP::first(wave, lane);  // the same of all of a wavefront's loads
      d.row = t.row0;
      d.at = (uint32_t)x * kSize | none_if(x >= p.k_in);
      if (!gathered)
#pragma unroll
        for (int i = 0; i < G::kPL; ++i)
          d.P.off[i] =
              d.at + (uint32_t)OpP::row(wave + G::kWaves * i, lane) * (uint32_t)ld * kSize;
    }
    if constexpr (OP == kMmWgrad) {
      d.Q.base = g + (uint64_t)(t.row0 * p.ldg * kSize);
#pragma unroll
      for (int i = 0; i < G::kQL; ++i) {
        const int l = wave + G::kWaves * i, x = OpQ::first(l, lane);
        const uint32_t c = OpQ::row(l, lane);
        d.Q.off[i] = (c * (uint32_t)p.ldg + t.j0 + x) * kSize | none_if(x >= t.nrows);
      }
    } else {
      const int64_t ld = OP == kMmForward ? p.lda : p.ldg;
      const bool gathered = OP == kMmForward && p.src;
      d.Q.base = (OP == kMmForward ? a : g) + (gathered ? 0 : (uint64_t)(t.row0 * ld * kSize));
#pragma unroll
      for (int i = 0; i < G::kQL; ++i) {
        const int l = wave + G::kWaves * i, x = OpQ::row(l, lane);
        uint32_t r = x;
        if constexpr (OP == kMmForward)
          if (gathered) r = act_row(p, d.route[i]);
        d.Q.off[i] = (r * (uint32_t)ld + OpQ::first(l, lane)) * kSize | none_if(x >= t.nrows);
      }
    }
    place(d);
  }
  // What changes from stage to stage besides the bases: gathered rows, and the last stage's end.
  __device__ __forceinline__ void place(Loads& d) const {
    if (OP == kMmWgrad && p.src) {
      constexpr int kRows = OP == kMmWgrad ? OpP::kRows : 1;
      const int h = here(lane) / OpP::kLanes;
#pragma unroll
      for (int i = 0; i < G::kPL; ++i) {
        uint32_t at = 0;
#pragma unroll
        for (int x = 0; x < kRows; ++x) {
          const uint32_t r =
              (uint32_t)act_row(p, d.route[(i * kRows + x) % (sizeof(d.route) / 4)]) *
              (uint32_t)p.lda * 2;
          at = h == x ? r : at;
        }
        d.P.off[i] = d.at + at;
      }
    }
    if (d.left < kC) {
      d.P.mask(d.left, wave, here(lane));
      d.Q.mask(d.left, wave, here(lane));
    }
  }

  // Load i of the next stage to the buffer at `at`, P's first.
  static constexpr int kLoads = G::kPL + G::kQL;
  __device__ __forceinline__ void issue(const Loads& d, int i, uint32_t at) const {
    if (i < G::kPL)
      d.P.issue(i, at, wave);
    else
      d.Q.issue(i - G::kPL, at + G::BI * kC * 2, wave);
  }
  // The tiles that the loads walk through, ahead of the products.
  struct Walk {
    uint32_t q, step, end;
    Tile next;  // where the loads go after the tile that they are in
  };
  // From the stage whose loads are out to the next; what the one after it needs is fetched.
  __device__ __forceinline__ void advance(Loads& d, Walk& k) const {
    d.left -= kC;
    if (d.left > 0) {
      if constexpr (OP == kMmForward) {
        d.P.base += kC * 2;
        d.Q.base += kC * 2;
      } else if constexpr (OP == kMmDgrad) {
        d.P.base += (uint64_t)kC * p.k_in * 2;
        d.Q.base += kC * 2;
      } else {
        d.Q.base += (uint64_t)(kC * p.ldg * 2);
        if (!p.src) d.P.base += (uint64_t)(kC * p.lda * 2);
        d.row += kC;
      }
      place(d);
    } else {
      plan(d, k.next);
    }
    ahead(d, k);
  }
  __device__ __forceinline__ void ahead(Loads& d, Walk& k) const {
    if (d.left <= kC) {  // the next stage is another tile's
      k.q += k.step;
      if (k.q < k.end) {
        k.next = find(k.q);
        fetch(d, k.next, k.next.row0, k.next.nc);
      } else {
        k.next.nc = 0;  // a tile of nothing: its loads fetch nothing
      }
    } else if (OP == kMmWgrad) {
      fetch(d, k.next, d.row + kC, d.left - kC);
    }
  }

  // ---- results ----
  typedef __attribute__((address_space(3))) v4f* pv4f;
  // What the results of a wavefront's 64 i's by 32 j's (rows j0 .. of the tile) are joined with: the
  // residual, or gate and up.  All is read at once, from the nearest place there is.
  static constexpr bool kZ = OP == kMmDgrad && SWIGLU;
  static constexpr bool kResidual = OP == kMmForward && !SWIGLU;
  static constexpr int XDT = kZ ? DT : ODT;
  typedef typename Elem<XDT>::type X4 __attribute__((ext_vector_type(4)));
  struct Extra {
    X4 a[kZ || kResidual ? 8 : 1], b[kZ ? 8 : 1];
  };
  __device__ __forceinline__ void read_extra(Extra& x, const Tile& t, int j0) const {
    const int lane = here(this->lane);
    const int rows = max(min(t.nrows - j0, 32), 1);
    const int i = min(t.i0 + wi * 64 + (lane & 15) * 4, ni() - 4);
    const int64_t row0 = (int64_t)t.row0 + min(j0, t.nrows - 1);
    const typename Elem<XDT>::type* from =
        static_cast<const typename Elem<XDT>::type*>(kZ ? p.z : p.residual);
    const int64_t ld = kZ ? p.ldz : p.ldres;
    if (!kZ && !(kResidual && p.residual)) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t at = (row0 + min(4 * k + lane / 16, rows - 1)) * ld + i;
      x.a[kZ || kResidual ? k : 0] = *reinterpret_cast<const X4*>(from + at);
      if constexpr (kZ) x.b[k] = *reinterpret_cast<const X4*>(from + at + p.k_in);
    }
  }
  // The lane's bias: of its 4 i's, or of its 4 gates and ups.
  struct Bias {
    v4f a, b;
  };
  __device__ __forceinline__ Bias read_bias(const Tile& t) const {
    Bias x = {};
    if (OP == kMmForward && p.bias) {
      const int lane = here(this->lane);
      const int i = t.i0 + wi * (kGates ? 32 : 64) + (lane & (kGates ? 7 : 15)) * 4;
      const int64_t at = (int64_t)t.expert * p.n_out * (kGates ? 2 : 1) + min(i, p.n_out - 4);
      x.a = load4<DT>(p.bias, at);
      if (kGates) x.b = load4<DT>(p.bias, at + p.n_out);
    }
    return x;
  }
  __device__ static v4f wide(const X4& x) {
    return (v4f){(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
  }

  // They are turned in 4 KB of LDS, 16 rows at a time, so that 16 lanes hold 64 neighbouring i's of
  // a row.
  __device__ __forceinline__ void finish(const Tile& t, const v16f& a0, const v16f& a1, int j0,
                                         uint32_t turn, const Extra& x,
                                         const Bias& bias) const {
    const int lane = here(this->lane);
    const int rows = min(t.nrows - j0, 32);
    const int64_t row0 = (int64_t)t.row0 + j0;
    auto put = [&](int half_rows) {
      const int l32 = lane & 31, half = lane >> 5;
      lanes_fence();
      if ((l32 >> 4) == half_rows) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int g = 0; g < 4; ++g) {  // i's 32 m + 8 g + 4 half + 0..3 of row l32
            const v16f& y = m ? a1 : a0;
            const int piece = 8 * m + 2 * g + half;
            *(pv4f)(uintptr_t)(turn + (l32 & 15) * 256 + 16 * (piece ^ (l32 & 15))) =
                (v4f){y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]};
          }
      }
      lanes_fence();
    };
    auto get = [&](int r, int piece) {
      return *(pv4f)(uintptr_t)(turn + (r & 15) * 256 + 16 * (piece ^ (r & 15)));
    };
    if constexpr (kGates) {
      const int i = t.i0 + wi * 32 + (lane & 7) * 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k % 2 == 0) put(k / 2);
        const int r = 8 * k + lane / 8;
        const v4f g = get(r, lane & 7) + bias.a, u = get(r, 8 + (lane & 7)) + bias.b;
        v4f h;
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = g[q] * sigmoid(g[q]) * u[q];
        if (r < rows && i < p.n_out) {
          if (p.z) {
            const int64_t at = (row0 + r) * p.ldz + i;
            store4<DT>(p.z, at, g);
            store4<DT>(p.z, at + p.n_out, u);
          }
          store4<ODT>(p.out, (row0 + r) * p.ldo + i, h);
        }
      }
    } else {
      const int i = t.i0 + wi * 64 + (lane & 15) * 4;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k % 4 == 0) put(k / 4);
        const int r = 4 * k + lane / 16;
        v4f y = get(r, lane & 15);
        const int64_t o = (row0 + r) * p.ldo + i;
        if constexpr (kZ) {
          v4f dg, du;
          swiglu_gradient(y, wide(x.a[k]), wide(x.b[k]), dg, du);
          if (r < rows && i < ni()) {
            store4<ODT>(p.out, o, dg);
            store4<ODT>(p.out, o + p.k_in, du);
          }
        } else {
          if constexpr (OP == kMmForward) {
            y += bias.a;
            if (p.residual) y += wide(x.a[k]);
          }
          if (r < rows && i < ni()) store4<ODT>(p.out, o, y);
        }
      }
    }
  }

  // wgrad: a wavefront's 32 j's (j0 ..) of 64 i's, rounded first if they are to be, through 4 KB.
  __device__ __forceinline__ void finish_own(const Tile& t, const v16f& a0, const v16f& a1, int j0,
                                             uint32_t turn) const {
    typedef typename Half<DT>::v4 v4h;
    typedef __attribute__((address_space(3))) v4h* pv4h;
    typedef __attribute__((address_space(3))) v4i* pv4i;
    const int lane = here(this->lane);
    const int l32 = lane & 31, half = lane >> 5, rows = min(t.nrows - j0, 32);
    constexpr int kSize = ODT == kF32 ? 4 : 2;
    constexpr int kTiles = ODT == kF32 ? 1 : 2;  // of 128 bytes a row
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<uint8_t*>(p.out) + ((int64_t)t.expert * p.n_out + t.j0 + j0) * p.k_in * kSize,
        0, (int)kNone, 0x00020000);
#pragma unroll
    for (int m0 = 0; m0 < 2; m0 += kTiles) {
      lanes_fence();
#pragma unroll
      for (int m = m0; m < m0 + kTiles; ++m)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const v16f& y = m ? a1 : a0;
          const v4f v = {y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]};
          if constexpr (ODT == kF32) {
            *(pv4f)(uintptr_t)(turn + l32 * 128 + 16 * ((2 * g + half) ^ (l32 & 7))) = v;
          } else {
            typedef typename Half<DT>::T T;
            const v4h h = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
            *(pv4h)(uintptr_t)(turn + l32 * 128 + 16 * ((4 * (m - m0) + g) ^ (l32 & 7)) +
                               8 * half) = h;
          }
        }
      lanes_fence();
      const int i = t.i0 + wi * 64 + m0 * 32 + (lane & 7) * (16 / kSize);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 8 * k + lane / 8;
        const v4i v = *(pv4i)(uintptr_t)(turn + r * 128 + 16 * ((lane & 7) ^ (r & 7)));
        // past the edges the offset is past the descriptor: each wavefront issues the same stores
        __builtin_amdgcn_raw_buffer_store_b128(
            __builtin_bit_cast(v4u, v), rsrc,
            ((r * p.k_in + i) * kSize) | none_if(r >= rows || i >= p.k_in), 0, 0);
      }
    }
  }

  // Bias gradient, in the tiles of the first i's: the sums of Q's columns over c.  A lane sums 4
  // columns of every kSumRows-th row of a stage.
  static constexpr int kSumLanes = G::BJ / 4, kSumRows = 64 / kSumLanes * G::kWaves;
  __device__ __forceinline__ void sum_columns(v4f& sum, uint32_t q) const {
    typedef __attribute__((address_space(3))) const typename Half<DT>::v4* pv4h;
    const int c0 = wave * (64 / kSumLanes) + lane / kSumLanes, l = lane % kSumLanes;
#pragma unroll
    for (int c = 0; c < kC; c += kSumRows) {  // kSumRows is a multiple of 4
      const typename Half<DT>::v4 v =
          *(pv4h)(uintptr_t)(q + (c + c0) * (G::BJ * 2) + (((l >> 3) ^ (c0 & 3)) * 64) + (l & 7) * 8);
#pragma unroll
      for (int x = 0; x < 4; ++x) sum[x] += (float)v[x];
    }
  }
  __device__ __forceinline__ void finish_sums(const Tile& t, const v4f& sum, uint32_t turn) const {
    barrier();  // the other wavefronts' results are turned there
    *(pv4f)(uintptr_t)(turn + ((wave * (64 / kSumLanes) + lane / kSumLanes) * G::BJ +
                               lane % kSumLanes * 4) * 4) = sum;
    barrier();
    if ((int)threadIdx.x * 4 < t.nrows) {
      v4f y = {};
#pragma unroll
      for (int r = 0; r < kSumRows; ++r)
        y += *(pv4f)(uintptr_t)(turn + (r * G::BJ + threadIdx.x * 4) * 4);
      store4<ODT>(p.bias_out, (int64_t)t.expert * p.n_out + t.j0 + threadIdx.x * 4, y);
    }
    barrier();
  }

  // ---- the walk ----
  __device__ __forceinline__ void run() {
    const uint32_t all = count();
    // Workgroups go to the 8 XCDs in turn.  Each XCD takes an eighth of the tiles, and its
    // workgroups walk through it side by side.
    const uint32_t xcd = blockIdx.x & 7, step = gridDim.x >> 3;
    const uint32_t end = (uint32_t)((uint64_t)all * (xcd + 1) >> 3);
    uint32_t q = (uint32_t)((uint64_t)all * xcd >> 3) + (blockIdx.x >> 3);
    if (q >= end) return;

    const uint32_t buf0 = __builtin_amdgcn_readfirstlane(lds_address(lds.buf[0]));
    Reader<G::BI, kC, G::TI, 1, kPWide> rp;
    Reader<G::BJ, kC, G::TJ, G::WJ, kQWide> rq;
    rp.plan(buf0, wi * G::TI, lane);
    rq.plan(buf0 + G::BI * kC * 2, wj, lane);

    const uint32_t own = buf0 + kBufs * G::kBuf;
    Loads d;
    Walk walk{q, step, end, find(q)};
    Tile t = walk.next;
    auto load_all = [&](uint32_t to) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) issue(d, i, to);
    };
    fetch(d, t, t.row0, t.nc);
    plan(d, t);
    ahead(d, walk);
    load_all(buf0);
    for (int s = 1; s < kBufs; ++s) {
      advance(d, walk);
      load_all(buf0 + s * G::kBuf);
    }
    // Stage s + 1 has landed when no more is out than the loads of the kBufs - 2 that followed it.
    constexpr int kKeep = (kBufs - 2) * kLoads;
    wait_and_barrier<kKeep + kLoads>();
    uint32_t buf = 0;  // the buffer of the stage at work, as an offset
    // Own turn: kBufs - 1 waits after a tile's stores are still for loads that went out before them.
    constexpr int kStores = G::TJ * (ODT == kF32 ? 8 : 4);
    int relaxed = 0;
    for (;;) {
      const int stages = max((t.nc + kC - 1) / kC, 1);
      const int row_tiles = (t.nrows + 31) / 32;
      const int live = row_tiles > wj ? (row_tiles - wj + G::WJ - 1) / G::WJ : 0;
      const bool sums = OP == kMmWgrad && p.bias_out && t.i0 == 0;
      v4f sum = {};
      auto go = [&](auto N) {
        constexpr int NL = decltype(N)::value, M = NL > 0 ? NL : 1;
        if constexpr (NL <= G::TJ) {
          if (live != NL) return;
          v16f acc[G::TI][M];
#pragma unroll
          for (int i = 0; i < G::TI; ++i)
#pragma unroll
            for (int j = 0; j < NL; ++j)
#pragma unroll
              for (int x = 0; x < 16; ++x) acc[i][j][x] = 0.0f;
          struct Ops {
            v4i p[G::TI], q[M];
          };
          auto read = [&](int s, uint32_t b) {
            Ops o;
            if constexpr (NL > 0) {
#pragma unroll
              for (int i = 0; i < G::TI; ++i) o.p[i] = rp.read(i, s, b);
#pragma unroll
              for (int j = 0; j < NL; ++j) o.q[j] = rq.read(j, s, b);
            }
            __builtin_amdgcn_sched_barrier(0);
            return o;
          };
          // The products of a step, with `first` after the first of them and a part of `loads` after
          // each.
          auto products = [&](const Ops& o, auto first, auto loads) {
            constexpr int kMany = NL * G::TI;
            if constexpr (kMany == 0) {
              first();
              loads(0, 1);
            }
#pragma unroll
            for (int m = 0; m < kMany; ++m) {
              const int i = m % G::TI, j = m / G::TI;
              acc[i][j] = mfma16<DT>(o.p[i], o.q[j], acc[i][j]);
              if (m == 0) first();
              loads(m, kMany);
            }
            __builtin_amdgcn_sched_barrier(0);
          };
          auto nothing = []() {};
          auto no_loads = [](int, int) {};
          Ops now = read(0, buf);
          // A stage's first operands are read in the last step of the one before, after the barrier
          // that ends the reads of that one; then its buffer is loaded again.
          auto stage = [&](auto LOAD) {
            const uint32_t other = (buf + G::kBuf) % (kBufs * G::kBuf);
            Ops then = read(1, buf);
            if constexpr (G::kSteps == 4) {
              products(now, nothing, no_loads);
              now = read(2, buf);
              products(then, nothing, no_loads);
              then = read(3, buf);
            }
            if constexpr (OP == kMmWgrad)
              if (sums) sum_columns(sum, buf0 + buf + G::BI * kC * 2);
            products(now, [&]() {
              __builtin_amdgcn_sched_barrier(0);
              advance(d, walk);
            }, no_loads);
            if (kOwnTurn && relaxed > 0) {
              wait_and_barrier<kKeep + kStores>();
              --relaxed;
            } else {
              wait_and_barrier<kKeep>();
            }
            now = read(0, other);
            if constexpr (decltype(LOAD)::value) {
              products(then, nothing, [&](int m, int many) {
#pragma unroll
                for (int l = m * kLoads / many; l < (m + 1) * kLoads / many; ++l)
                  issue(d, l, buf0 + buf);
                __builtin_amdgcn_sched_barrier(0);
              });
            } else {
              products(then, nothing, no_loads);
            }
            buf = other;
          };
          if constexpr (kOwnTurn) {
            int left = stages;
            do stage(std::true_type());
            while (--left > 0);
#pragma unroll
            for (int j = 0; j < NL; ++j)
              finish_own(t, acc[0][j], acc[1][j], (j * G::WJ + wj) * 32, own + 4096 * wave);
            relaxed = NL == G::TJ ? kBufs - 1 : 0;
          } else {
            // the results are turned in the buffer that the last stage was in
            for (int left = stages; left > 1; --left) stage(std::true_type());
            const uint32_t turn = buf0 + buf + 4096 * wave;
            stage(std::false_type());
            const Bias bias = read_bias(t);
            Extra x, next;
            if (NL > 0) read_extra(x, t, wj * 32);
#pragma unroll
            for (int j = 0; j < NL; ++j) {
              if (j + 1 < NL) read_extra(next, t, ((j + 1) * G::WJ + wj) * 32);
              finish(t, acc[0][j], acc[1][j], (j * G::WJ + wj) * 32, turn, x, bias);
              x = next;
            }
          }
        }
      };
      go(std::integral_constant<int, 0>{});
      go(std::integral_constant<int, 1>{});
      go(std::integral_constant<int, 2>{});
      go(std::integral_constant<int, 3>{});
      go(std::integral_constant<int, 4>{});
      static_assert(G::TJ <= 4, "instances");
      if (sums) finish_sums(t, sum, own);
      q += step;
      if (q >= end) break;
      if constexpr (!kOwnTurn) {
        barrier();
        load_all(buf0 + (buf + (kBufs - 1) * G::kBuf) % (kBufs * G::kBuf));
      }
      t = find(q);
    }
    // no load to LDS is under way when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  }
};

}  // namespace tile

}  // namespace moe
