// Tiles of products of int8 activations, in their own row-major order, with the
// 8-bit weights (w8.hip) or the two ternary weights of a gated block (gated.hip)
// on the int8 matrix cores: C[i][j] = sum_k q[i][k] * w[j][k], exact in int32.
//
// K goes in slabs of 128 (a gated block, whose weights are then 32 bytes a row) or
// of 64 (8-bit weights: of a 256 x 256 tile that is 32 KB, four of which fit LDS).
// Both operands go from global memory straight into a ring of buffers in LDS:
//   activations     rows of a slab's bytes; chunk c (16 bytes) of row r at chunk
//                   c ^ ((r / 2) & 7), or c ^ ((r / 4) & 3) of a slab of 64, so
//                   that the 16 rows that LDS serves together lie in distinct
//                   banks
//   weights         as they are stored: per block of 16 rows one kilobyte (8-bit)
//                   or half of one (ternary), [chunk][row][16 bytes], which 16 rows
//                   of an operand read without a conflict.  Ternary weights are
//                   expanded in registers (expand16)
// The weights are the matrix core's first operand, so that a lane's sums belong
// to one token: lane (lr, lg) = (lane % 32, lane / 32) holds, of a 32 x 32
// subtile, row lr at columns 8 a + 4 lg .. + 3 in elements 4 a .. 4 a + 3.
//
// What lies past K in the activations' rows is read (the last chunk again) and
// meets zeros of the weights' padding.  Rows past the end read the last one; their
// sums are not stored.
//
// What bounds a tile: of 256 x 256 the matrix cores, busy 55% of the cycles that a
// CU has work, at the clock that their power leaves (8-bit 2048 x 14336 x 4096: 117
// us, 2.06 POPS; on zeros 103); smaller ones the cache lines that a CU's L1 has in
// flight, some 70: about 24 bytes a cycle go to LDS whatever the tile, so a tile
// that needs fewer bytes a product is faster until it leaves CUs without work
// (codes_plan.hpp), and loads are whole lines where they can be (weights in the
// order of their storage in place of rows: 300 x 4096 x 14336 40 -> 35 us).
#pragma once

#include "codes_plan.hpp"
#include "common.hpp"
#include "internal.hpp"

#include <atomic>
#include <type_traits>

namespace bl {

typedef int32_t v16i __attribute__((ext_vector_type(16)));

struct CodesJob {
  const int8_t* q;  // rows of ldq bytes
  int32_t ldq;      // a multiple of 16, or of 4 (tiles that load WORDS)
  int32_t m, n, k;
  const uint8_t* w;
  int32_t ktiles, blocks;  // of the weights' storage
  int32_t slabs;           // ceil(k / the tile's slab)
  int32_t tiles_i, tiles_j;
  int32_t ksplit, kspw;  // parts of k, and slabs a part
  int32_t past_cache;    // the outputs are more than the L2 caches hold, and go past them
  int32_t* part;         // ksplit > 1: int32 sums [ksplit][m][ldp] (gated: [ksplit][2][m][ldp])
  int32_t ldp;           // part_pitch(n)
};

namespace codes_gemm {

__device__ __forceinline__ v16i mfma_32x32x32_i8(v4i a, v4i b, v16i c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Waits until at most `ahead` slabs of D loads each are still in flight.
template <int D, int C>
__device__ __forceinline__ void wait_slabs(int ahead) {
  if constexpr (C == 0) {
    wait_vm<0>();
  } else {
    if (ahead >= C)
      wait_vm<C * D>();
    else
      wait_slabs<D, C - 1>(ahead);
  }
}

__device__ __forceinline__ void dma16(const void* src, int8_t* lds_dst) {
  __builtin_amdgcn_global_load_lds((const BL_GLOBAL void*)src,
                                   (__attribute__((address_space(3))) void*)lds_dst, 16, 0, 0);
}

__device__ __forceinline__ void dma4(const void* src, int8_t* lds_dst) {
  __builtin_amdgcn_global_load_lds((const BL_GLOBAL void*)src,
                                   (__attribute__((address_space(3))) void*)lds_dst, 4, 0, 0);
}

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");  // no LDS access moves across
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace codes_gemm

// int8 values 64 u of the 16 weights of a dword of the gated storage, four a
// dword, in order.
__device__ __forceinline__ v4i expand16(uint32_t p) {
  v4i r;
  r.x = (int32_t)(p & 0xC0C0C0C0u);
  r.y = (int32_t)((p << 2) & 0xC0C0C0C0u);
  r.z = (int32_t)((p << 4) & 0xC0C0C0C0u);
  r.w = (int32_t)((p << 6) & 0xC0C0C0C0u);
  return r;
}

// A wave's bf16 outputs of 32 rows on their way to memory.  A lane has runs of
// four columns of one row; stored like that an instruction would touch 32 rows,
// 16 bytes of each.  A pass through LDS, in a part of the wave's own (the ring is
// done with), makes it whole rows: `cols` columns, 16 bytes a lane.
template <int COLS>
struct CodesRows {
  static constexpr int kPitch = 2 * COLS + 16;  // 16 bytes off: rows start at distinct banks
  static constexpr int kBytes = 32 * kPitch;
  static constexpr int LPR = COLS / 8, RPI = 64 / LPR;  // lanes a row, rows an instruction

  int8_t* mine;
  __device__ __forceinline__ explicit CodesRows(int8_t* lds) : mine(lds) {}

  // Columns c .. c + 3 (of the 32 rows' COLS) of row lr.
  __device__ __forceinline__ void put(int lr, int c, uint32_t lo, uint32_t hi) const {
    typedef int32_t v2i __attribute__((ext_vector_type(2)));
    *reinterpret_cast<v2i*>(mine + lr * kPitch + 2 * c) = v2i{(int32_t)lo, (int32_t)hi};
  }
  // Rows m0 .. m0 + 31 at columns n0 ... of out [m][n]; what is past them is not stored.
  __device__ __forceinline__ void store(uint16_t* out, int m0, int n0, int m, int n, bool past_cache) const {
    const int lane = threadIdx.x & 63;
    const int c = n0 + 8 * (lane % LPR);
    const bool wide = (n & 7) == 0;  // output rows are 16-byte aligned
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < 32 / RPI; ++q) {
      const int r = q * RPI + lane / LPR;
      const v4i v = *reinterpret_cast<const v4i*>(mine + r * kPitch + 16 * (lane % LPR));
      if (m0 + r >= m) continue;
      uint16_t* row = out + (int64_t)(m0 + r) * n;
      if (wide && c < n) {
        if (COLS >= 64 && past_cache) {
          // fenced: the compiler would make one store of the two branches', a plain one
          asm volatile("" ::: "memory");
          __builtin_nontemporal_store(v, G(reinterpret_cast<v4i*>(row + c)));
          asm volatile("" ::: "memory");
        } else {
          *G(reinterpret_cast<v4i*>(row + c)) = v;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < n) *G(row + c + e) = (uint16_t)((uint32_t)v[e >> 1] >> (16 * (e & 1)));
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
};

// One tile of TI tokens x TJ weight rows by WI x WJ waves.  TERNARY: the first
// half of the TJ rows is the gate's, the second the up projection's of the same
// TJ / 2 outputs, and so is each wave's share.  WORDS: activations are loaded four
// bytes a lane, from rows of any multiple of that, in place of 16.
template <int TI_, int TJ_, int WI_, int WJ_, int NST_, bool TERNARY, bool WORDS = false>
struct CodesTile {
  static constexpr int SL = TERNARY ? 128 : 64;        // k of a slab
  static constexpr int CA = SL / 16;                   // chunks of a row of activations or 8-bit weights
  static constexpr int kRowB = TERNARY ? SL / 4 : SL;  // bytes of a row of weights
  static constexpr int kSwzA = 16 / CA;  // rows in a row of banks
  static __device__ __forceinline__ int swz(int r, int c) { return c ^ ((r / kSwzA) & (CA - 1)); }
  static constexpr int TI = TI_, TJ = TJ_, WI = WI_, WJ = WJ_, NST = NST_, NW = WI * WJ;
  static constexpr int FI = TI / WI / 32, FJ = TJ / WJ / 32;
  static constexpr int kStage = TI * SL + TJ * kRowB;
  static constexpr int kLds = NST * kStage;
  static constexpr int kLoadA = WORDS ? 256 : 1024;  // bytes of a load of activations
  static constexpr int DA = TI * SL / kLoadA / NW;   // loads of a slab, per wave
  static constexpr int CB = TJ * kRowB / 1024;  // of the weights, all waves
  static constexpr int DB = CB < NW ? 1 : CB / NW;
  static constexpr int D = DA + DB;
  static constexpr int kCols = TERNARY ? TJ / 2 : TJ;  // outputs of a tile
  using Rows = CodesRows<kCols / WJ>;                  // a wave's outputs
  static_assert(NW * Rows::kBytes <= kLds, "they fit the ring");
  static_assert(DA * kLoadA * NW == TI * SL && (NST - 1) * D < 64 && (DB * NW == CB || NW % CB == 0), "whole loads");
  static_assert(FI * WI * 32 == TI && FJ * WJ * 32 == TJ && (!TERNARY || FJ % 2 == 0), "whole subtiles");

  // First row and (outputs') first column of the wave's share.
  static __device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }
  static __device__ __forceinline__ int row0() { return (wave() % WI) * (TI / WI); }
  static __device__ __forceinline__ int col0() { return (wave() / WI) * (kCols / WJ); }
  // Weight row (of the tile) of fragment j.
  static __device__ __forceinline__ int brow(int j) {
    if constexpr (TERNARY) return (j < FJ / 2 ? 0 : TJ / 2) + col0() + 32 * (j % (FJ / 2));
    return col0() + 32 * j;
  }

  static __device__ __forceinline__ void run(const CodesJob& J, int ti, int tj, int kp, int8_t* smem,
                                             v16i (&acc)[FI][FJ]) {
    using namespace codes_gemm;
    const int lane = threadIdx.x & 63, wv = wave();
    const int lr = lane & 31, lg = lane >> 5;
    const int i0 = ti * TI, wi0 = row0();
    const int s0 = kp * J.kspw, nsl = min(J.slabs - s0, J.kspw);
    const int blk0 = tj * (kCols / 16);

    // Per lane the offsets of a load's row and of its chunk in the slab.
    uint32_t ar[WORDS ? 1 : DA], ac[WORDS ? 1 : DA], br[DB];
    const uint32_t row_end = tile_last_row(TI, J.m - i0, J.ldq);
    if constexpr (WORDS) {  // of load 0 of wave 0, without the swizzle, which is one of the load
      ar[0] = (uint32_t)(lane / (SL / 4)) * (uint32_t)J.ldq;
      ac[0] = 4 * (lane % (SL / 4));
    }
#pragma unroll
    for (int i = 0; i < (WORDS ? 0 : DA); ++i) {
      const int pos = (wv * DA + i) * 64 + lane, r = pos / CA;
      ar[i] = (uint32_t)min(r, J.m - 1 - i0) * (uint32_t)J.ldq;
      ac[i] = 16 * swz(r, pos % CA);
    }
#pragma unroll
    for (int i = 0; i < DB; ++i) {  // waves past the last piece load one again, so that all wait alike
      const int pos = ((wv % CB) * DB + i) * 64 + lane;
      if constexpr (TERNARY) {
        const int b = pos >> 5, up = b >= TJ / 32;  // 512 bytes a block of 16 rows
        br[i] = (uint32_t)min(b - up * (TJ / 32), J.blocks - 1 - blk0) * ((uint32_t)J.ktiles * 2048) + 1024 * up +
                16 * (pos & 31);
      } else {
        br[i] = (uint32_t)min(pos >> 6, J.blocks - 1 - blk0) * ((uint32_t)J.ktiles * 1024) + 16 * (pos & 63);
      }
    }
    const int8_t* pa = J.q + (int64_t)i0 * J.ldq;
    const uint8_t* pb = J.w + (int64_t)blk0 * J.ktiles * (TERNARY ? 2048 : 1024);
    int next = s0;  // the slab that is loaded next
    // Load d (of D) of the next slab into the buffer st.
    auto issue_one = [&](int d, int8_t* st) {
      if (WORDS && d < DA) {
        const int l = wv * DA + d;
        const uint32_t row = min(ar[0] + (uint32_t)(l * (256 / SL)) * (uint32_t)J.ldq, row_end);
        const uint32_t last = (uint32_t)(J.ldq - 4 - next * SL);  // the row's last word for those past it
        dma4(pa + (int64_t)next * SL + row + min(ac[0] ^ (uint32_t)(16 * (l & (CA - 1))), last), st + l * 256);
      } else if (d < DA) {
        // the row's last chunk for those past it
        const uint32_t last = (uint32_t)(J.ldq - 16 - next * SL);
        dma16(pa + (int64_t)next * SL + ar[d] + min(ac[d], last), st + (wv * DA + d) * 1024);
      } else {
        const int e = d - DA;
        int8_t* dst = st + TI * SL + ((wv % CB) * DB + e) * 1024;
        if constexpr (TERNARY) {
          dma16(pb + (int64_t)(next >> 1) * 2048 + 512 * (next & 1) + br[e], dst);  // two slabs a tile
        } else {
          dma16(pb + (int64_t)next * 1024 + br[e], dst);
        }
      }
      if (d == D - 1) ++next;
    };

#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

    constexpr int KS = SL / 32;
    // Fragments of step ks of a slab: 32 k, 16 a lane half (chunk 2 ks + lg of a
    // row; TERNARY: chunk 4 lg + ks, dword ks of the weights' chunk lg).
    v4i fa[2][FI], fb[2][FJ], cj[FJ];
    const int8_t* sa = smem;  // the current slab's buffer
    auto load = [&](int ks, v4i (&a)[FI], v4i (&b)[FJ]) {
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        const int r = wi0 + 32 * i + lr, c = TERNARY ? KS * lg + ks : 2 * ks + lg;
        a[i] = *reinterpret_cast<const v4i*>(sa + SL * r + 16 * swz(r, c));
      }
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int r = brow(j) + lr;
        const int8_t* sb = sa + TI * SL + 16 * kRowB * (r >> 4) + 16 * (r & 15);
        if constexpr (!TERNARY)
          b[j] = *reinterpret_cast<const v4i*>(sb + 256 * (2 * ks + lg));
        else if (ks == 0)
          b[j] = *reinterpret_cast<const v4i*>(sb + 256 * lg);
      }
    };
    // Products of step ks.  `mid` runs behind the first of them, which waits for the
    // step's fragments: what it reads from LDS then has the other products' time
    // to arrive.  With ISSUE, a load of the slab that goes to `st` between any two.
    auto multiply = [&](auto issue, int ks, const v4i (&a)[FI], const v4i (&b)[FJ], int8_t* st, const auto& mid) {
      constexpr bool ISSUE = decltype(issue)::value;
      constexpr int P = FI * FJ;
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        v4i w;
        if constexpr (TERNARY)
          w = expand16((uint32_t)cj[j][ks]);
        else
          w = b[j];
#pragma unroll
        for (int i = 0; i < FI; ++i) {
          acc[i][j] = mfma_32x32x32_i8(w, a[i], acc[i][j]);
          if (i + j == 0) {
            __builtin_amdgcn_sched_barrier(0);
            mid();
            __builtin_amdgcn_sched_barrier(0);
          }
          if constexpr (ISSUE) {
#pragma unroll
            for (int d = 0; d < D; ++d)
              if (d * P / D == j * FI + i) {
                __builtin_amdgcn_sched_barrier(0);
                issue_one(d, st);
                __builtin_amdgcn_sched_barrier(0);
              }
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int p = 0; p < NST; ++p)
      if (p < nsl) {
#pragma unroll
        for (int d = 0; d < D; ++d) issue_one(d, smem + p * kStage);
      }
    wait_slabs<D, NST - 1>(min(nsl - 1, NST - 1));
    barrier();
    load(0, fa[0], fb[0]);
    int buf = 0;
    // A slab.  Behind the first product of its last step its fragments are all in
    // registers: when every wave is there, its buffer is free.  The next slab's
    // first fragments are then read, and the buffer refilled between the products.
    auto slab = [&](auto issue, int s) {
      constexpr bool ISSUE = decltype(issue)::value;
      if constexpr (TERNARY) {
#pragma unroll
        for (int j = 0; j < FJ; ++j) cj[j] = fb[0][j];
      }
#pragma unroll
      for (int ks = 0; ks < KS - 1; ++ks) {
        auto ahead = [&]() { load(ks + 1, fa[(ks + 1) & 1], fb[(ks + 1) & 1]); };
        multiply(std::false_type{}, ks, fa[ks & 1], fb[ks & 1], nullptr, ahead);
      }
      int8_t* st = smem + buf * kStage;
      auto turn = [&]() {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slab's LDS reads are done
        if (ISSUE || s + 1 < nsl) {
          wait_vm<ISSUE ? (NST - 2) * D : 0>();
          barrier();
          buf = buf + 1 == NST ? 0 : buf + 1;
          sa = smem + buf * kStage;
          load(0, fa[0], fb[0]);
        }
      };
      multiply(issue, KS - 1, fa[(KS - 1) & 1], fb[(KS - 1) & 1], st, turn);
    };
    int s = 0;
    for (; s + NST < nsl; ++s) slab(std::true_type{}, s);
    for (; s < nsl; ++s) slab(std::false_type{}, s);
  }
};

// Workgroups go to the 8 XCDs round-robin and each has its own L2, so each XCD
// takes one contiguous share of the tiles, walked in groups of up to four tile
// rows so that neighbours in time share operands both ways.
__device__ __forceinline__ bool codes_tile_of(int l, const CodesJob& J, int* ti, int* tj, int* kp) {
  const int T = J.tiles_i * J.tiles_j * J.ksplit, chunk = (T + 7) >> 3;
  const int w = l >> 3;
  int t = (l & 7) * chunk + w;
  if (w >= chunk || t >= T) return false;
  const int per = J.tiles_i * J.tiles_j;
  *kp = t / per;
  t -= *kp * per;
  const int g = t / (4 * J.tiles_j), rows = min(4, J.tiles_i - 4 * g);
  t -= g * 4 * J.tiles_j;
  *ti = 4 * g + t % rows;
  *tj = t / rows;
  return true;
}

// Up to eight bf16 outputs of one row from column n on.
__device__ __forceinline__ void codes_put8(uint16_t* row, int n, int cols, bool wide, const uint32_t* w) {
  if (wide && n + 8 <= cols) {
    *G(reinterpret_cast<v4i*>(row + n)) = v4i{(int32_t)w[0], (int32_t)w[1], (int32_t)w[2], (int32_t)w[3]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < cols) *G(row + n + e) = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// int32 sums of a part (32 x 32 subtile: one row a lane).  Rows of parts are of
// whole eights of columns, `ldp`; the ones past N are sums of the last blocks again.
__device__ __forceinline__ void codes_put_part(int32_t* row, int n0, int ldp, const v16i& acc) {
  const int lg = (threadIdx.x >> 5) & 1;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int n = n0 + 8 * a + 4 * lg;
    if (n < ldp)
      *G(reinterpret_cast<v4i*>(row + n)) = v4i{acc[4 * a], acc[4 * a + 1], acc[4 * a + 2], acc[4 * a + 3]};
  }
}

// Adds eight columns' sums of the parts, in order, four parts' loads at a time.
__device__ __forceinline__ void codes_add_parts(const int32_t* src, int64_t slice, int ksplit, int32_t (&v)[8]) {
  for (int p = 0; p < ksplit; p += 4) {
    v4i t[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        t[u][h] = p + u < ksplit ? *G(reinterpret_cast<const v4i*>(src + (p + u) * slice + 4 * h)) : v4i{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += t[u][e >> 2][e & 3];
  }
}

// Activations whose rows do not start at a multiple of 16 bytes, in rows that do
// (K rounded up to 16, the rest zeros): 16 bytes a thread.
static __global__ __launch_bounds__(256) void codes_pad_kernel(const int8_t* __restrict__ q, int64_t total,
                                                                int32_t k, int32_t ldq, int8_t* __restrict__ out) {
  const int cpr = ldq >> 4;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
    const int64_t m = id / cpr;
    const int c = 16 * (int)(id - m * cpr);
    v4i v;
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] = c + 4 * d < k ? *G(reinterpret_cast<const int32_t*>(q + m * k + c + 4 * d)) : 0;
    *G(reinterpret_cast<v4i*>(out + 16 * id)) = v;
  }
}

inline hipError_t codes_pad(const int8_t* q, int64_t m, int64_t k, int32_t ldq, int8_t* out, hipStream_t s) {
  const int64_t total = m * (ldq >> 4), grid = (total + 255) / 256;
  codes_pad_kernel<<<(unsigned)(grid < 65536 ? grid : 65536), 256, 0, s>>>(q, total, (int32_t)k, ldq, out);
  return hipGetLastError();
}

// Outputs of more than the eight L2 caches' 32 MB: kept there they would push out the
// operands, and be written back at the kernel's end (8-bit 2048 x 14336 x 4096: 141
// -> 128 us).  Rows of a wave shorter than a cache line are stored plainly.
inline int32_t codes_past_cache(int64_t m, int64_t n) { return 2 * m * n > (int64_t(32) << 20) ? 1 : 0; }

// Columns of a row of a part.
inline int64_t part_pitch(int64_t n) { return round_up(n, 8); }

inline void set_plan(CodesJob& J, const CodesPlan& p, int32_t* part) {
  J.past_cache = codes_past_cache(J.m, J.n);
  J.slabs = p.slabs;
  J.tiles_i = p.tiles_i;
  J.tiles_j = p.tiles_j;
  J.ksplit = p.ksplit;
  J.kspw = p.kspw;
  J.part = part;
  J.ldp = (int32_t)part_pitch(J.n);
}

// Launches a kernel with `lds` bytes of dynamic LDS, of at most `most`: an attribute
// above 64 KB, set once per device and kernel (`done` is the caller's).
template <typename Kernel, typename Args>
hipError_t codes_launch(Kernel kernel, std::atomic<bool>* done, dim3 grid, unsigned threads, size_t lds, size_t most,
                        hipStream_t s, const Args& args) {
  if (lds > 64 * 1024) {
    const int dev = current_device_index();
    if (!done[dev].load(std::memory_order_acquire)) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)most);
      if (e != hipSuccess) return e;
      done[dev].store(true, std::memory_order_release);
    }
  }
  kernel<<<grid, threads, lds, s>>>(args);
  return hipGetLastError();
}

}  // namespace bl
