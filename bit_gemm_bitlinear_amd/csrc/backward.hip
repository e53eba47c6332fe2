// Gradients of BitLinear from its 8-bit activation checkpoint.
//
//   dx[m][k] = bf16( sum_n dy[m][n] * u[n][k] / w_scale )
//   dw[n][k] = sum_m dy[m][n] * xhat[m][k],  xhat = bf16(q / x_scale)
//   db[n]    = sum_m dy[m][n]
//
// Both are matrix products C[i][j] = sum_c A[i][c] B[j][c].  u in {-1, 0, 1}
// and xhat are bf16 values, so every product is exact on the bf16 matrix cores
// and the sums are fp32.  A call is two launches (three where a product's c is
// split): one prepares the operands, one multiplies, dx and dw in one grid.
//
// Operands (prepare_kernel, in the workspace).  A matrix-core operand wants
// its c contiguous, which for dw is the token index and for the weights of dx
// the output index: both stored the other way round.  Each operand is kept as
// slabs of 64 c, [slab][row][64], zero-padded: a tile's slab is then one
// contiguous piece of memory whatever the row count (rows at a power-of-two
// stride would all fall on the same cache channels), 128 bytes a row:
//   dy  as A of dx: rows m, c = n;    dy^T as A of dw: rows n, c = m
//   xhat^T as B of dw: rows k, c = m (bf16)
//   u^T as B of dx: rows k, c = n, two bits a weight (16 bytes a row and slab)
#include "../../include/bitlinear_layer.h"
#include "backward_plan.hpp"
#include "common.hpp"
#include "internal.hpp"
#include "layer_internal.hpp"
#include "restore.hpp"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace bl {

namespace {

constexpr int kRow = 2 * kSlab;  // bytes of a bf16 row of a slab
constexpr int kCodes = kSlab / 4;  // bytes of a two-bit row of a slab

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int32_t v2i __attribute__((ext_vector_type(2)));
typedef v4i v4i_any __attribute__((aligned(2)));  // 16 bytes at any even address
typedef v2i v2i_any __attribute__((aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v16f mfma_32x32x16(v4i a, v4i b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a),
                                                 __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Operands

struct PrepArgs {
  int32_t begin[3];  // first workgroup of: dy, xhat, weights
  int64_t m, n, k;
  const uint16_t* dy;
  uint16_t* dys;  // [ceil(n/64)][m][64], or nullptr (no dx)
  uint16_t* dyt;  // [ceil(m/64)][n][64], or nullptr (no dw)
  float* dbp;     // [ceil(m/64)][n] sums over the slab's tokens, or nullptr
  const int8_t* q;
  const float* x_scale;
  uint16_t* xt;  // [ceil(m/64)][k][64]
  const uint8_t* packed;
  int32_t tiled;
  uint8_t* ut;  // [ceil(n/64)][k][16]
};

// Column j of eight rows of eight bf16 values: a byte select per pair of rows.
__device__ __forceinline__ v4i column8(const v4i (&r)[8], int j) {
  v4i o;
#pragma unroll
  for (int p = 0; p < 4; ++p)
    o[p] = (int32_t)__builtin_amdgcn_perm((uint32_t)r[2 * p + 1][j >> 1], (uint32_t)r[2 * p][j >> 1],
                                          (j & 1) ? 0x07060302u : 0x05040100u);
  return o;
}

// Eight rows of eight columns of dy [m][n] from (m0, n) on; what lies outside
// is zeros.
__device__ __forceinline__ void load_dy8(const uint16_t* __restrict__ dy, int64_t m, int64_t cols, int64_t m0,
                                         int64_t n, v4i (&r)[8]) {
  const int mv = (int)min((int64_t)8, m - m0);   // rows of the eight that exist (may be <= 0)
  const int nv = (int)min((int64_t)8, cols - n);  // columns
  if (nv >= 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // rows start at any even address; missing ones read the last
      const v4i v = *G(reinterpret_cast<const v4i_any*>(dy + min(m0 + i, m - 1) * cols + n));
      r[i] = i < mv ? v : v4i{0, 0, 0, 0};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v4i{0, 0, 0, 0};
    // the row's last columns, fewer than eight: one column of the eight rows a turn
#pragma unroll 1
    for (int e = 0; e < nv; ++e) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = *G(dy + min(m0 + i, m - 1) * cols + n + e);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h)
          r[i][h] |= (int32_t)((e >> 1) == h && i < mv ? v[i] << (16 * (e & 1)) : 0u);
    }
  }
}

// Eight rows of eight codes of q [m][k] from (m0, k0) on, restored to bf16, in
// rows; what lies outside is zeros (K % 4 == 0: four columns or eight).
struct Codes8 {
  v2i c[8];
  float xs[8];
};
__device__ __forceinline__ void load_codes8(const int8_t* __restrict__ q, const float* __restrict__ x_scale,
                                            int64_t m, int64_t cols, int64_t m0, int64_t k, Codes8& o) {
  const bool second = k + 4 < cols;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o.c[i] = v2i{0, 0};
    o.xs[i] = 1.0f;
    if (m0 + i >= m || k >= cols) continue;
    const int8_t* p = q + (m0 + i) * cols + k;
    o.c[i].x = *G(reinterpret_cast<const int32_t*>(p));
    if (second) o.c[i].y = *G(reinterpret_cast<const int32_t*>(p + 4));
    o.xs[i] = *G(x_scale + m0 + i);
  }
}
__device__ __forceinline__ void restore8(const Codes8& o, v4i (&r)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const RestoreRow d = restore_row(o.xs[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[i][e] = (int32_t)restore2((uint32_t)o.c[i][e >> 1], 2 * (e & 1), d);
  }
}

// Sums over eight rows of each of the eight columns.
__device__ __forceinline__ float column_sum8(const v4i (&r)[8], int e) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = (uint32_t)r[i][e >> 1];
    s += __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  return s;
}

// A thread's 8 tokens x 8 columns; a workgroup's 64 tokens x 256 columns.
// Eight lanes side by side hold one row's 64 columns on the way in and one
// column's 64 tokens on the way out: 128-byte pieces both ways.
__device__ __forceinline__ void prepare_dy(const PrepArgs& A, int wg) {
  const int cols = (int)((A.n + 255) >> 8);
  const int64_t ms = wg / cols, n0 = (int64_t)(wg - (int)ms * cols) * 256;
  const int mi = threadIdx.x & 7, ni = threadIdx.x >> 3;
  const int64_t m0 = ms * 64 + 8 * mi, n = n0 + 8 * ni;
  const int mv = (int)min((int64_t)8, A.m - m0);  // rows of the eight that exist (may be <= 0)
  v4i r[8];
  load_dy8(A.dy, A.m, A.n, m0, n, r);
  if (A.dys && n < ((A.n + 63) & ~(int64_t)63)) {
    uint16_t* d = A.dys + ((n >> 6) * A.m + m0) * 64 + (n & 63);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < mv) *G(reinterpret_cast<v4i*>(d + 64 * i)) = r[i];
  }
  if (A.dbp) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s = column_sum8(r, e);
      s += __shfl_xor(s, 1);
      s += __shfl_xor(s, 2);
      s += __shfl_xor(s, 4);
      if (mi == e && n + e < A.n) *G(A.dbp + ms * A.n + n + e) = s;
    }
  }
  if (A.dyt) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n + j < A.n) *G(reinterpret_cast<v4i*>(A.dyt + (ms * A.n + n + j) * 64 + 8 * mi)) = column8(r, j);
  }
}

__device__ __forceinline__ void prepare_xhat(const PrepArgs& A, int wg) {
  const int cols = (int)((A.k + 255) >> 8);
  const int64_t ms = wg / cols, k0 = (int64_t)(wg - (int)ms * cols) * 256;
  const int mi = threadIdx.x & 7, ki = threadIdx.x >> 3;
  const int64_t m0 = ms * 64 + 8 * mi, k = k0 + 8 * ki;
  if (k >= A.k) return;
  Codes8 c;
  load_codes8(A.q, A.x_scale, A.m, A.k, m0, k, c);
  v4i r[8];
  restore8(c, r);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (k + j < A.k) *G(reinterpret_cast<v4i*>(A.xt + (ms * A.k + k + j) * 64 + 8 * mi)) = column8(r, j);
}

// Two-bit transpose: a thread takes 16 weights k of 16 rows n (a dword each)
// to 16 dwords of 16 n, one per k, by four rounds of exchanges of ever
// smaller blocks.  In the result the codes of n = 2a and n = 2a + 1 sit at bits
// 2a and 16 + 2a (the rows are loaded in that order), where the product's
// expansion takes them as pairs.  Rows past N are code 1 (u = 0).
__device__ __forceinline__ void prepare_weights(const PrepArgs& A, int wg) {
  const int cols = (int)((A.k + 1023) >> 10);
  const int64_t slab = wg / cols;
  const int d = threadIdx.x & 3;
  const int64_t k = (int64_t)(wg - (int)slab * cols) * 1024 + 16 * (threadIdx.x >> 2);
  if (k >= A.k) return;
  const int64_t n0 = slab * 64 + 16 * d, rb = A.k >> 2, o = k >> 2;
  uint32_t w[16];
  // Every load unconditional: rows past N read the last one (and become code
  // 1), a row's last dword is read up to its end and shifted into place.
  if (rb >= 4) {
    const int64_t oc = min(o, rb - 4);
    const int sh = 8 * (int)(o - oc);
#pragma unroll
    for (int p = 0; p < 16; ++p) {
      const int64_t n = min(n0 + (p < 8 ? 2 * p : 2 * (p - 8) + 1), A.n - 1);
      const int64_t at = A.tiled ? tiled_chunk_offset(n, o & ~(int64_t)15, rb) + (o & 15) : n * rb + oc;
      w[p] = *G(reinterpret_cast<const u32_any*>(A.packed + at));
    }
#pragma unroll
    for (int p = 0; p < 16; ++p) w[p] >>= sh;
  } else {
#pragma unroll
    for (int p = 0; p < 16; ++p) {
      const int64_t n = min(n0 + (p < 8 ? 2 * p : 2 * (p - 8) + 1), A.n - 1);
      w[p] = 0;
#pragma unroll
      for (int b = 0; b < 3; ++b) w[p] |= (uint32_t)*G(A.packed + n * rb + min((int64_t)b, rb - 1)) << (8 * b);
    }
  }
#pragma unroll
  for (int p = 0; p < 16; ++p)
    if (n0 + (p < 8 ? 2 * p : 2 * (p - 8) + 1) >= A.n) w[p] = 0x55555555u;
#pragma unroll
  for (int h = 8; h >= 1; h >>= 1) {
    // exchange the upper half of each 2h-block of row p with the lower of row p + h
    const uint32_t mask = h == 8 ? 0x0000FFFFu : (h == 4 ? 0x00FF00FFu : (h == 2 ? 0x0F0F0F0Fu : 0x33333333u));
#pragma unroll
    for (int p = 0; p < 16; ++p) {
      if (p & h) continue;
      const uint32_t t = ((w[p] >> (2 * h)) ^ w[p + h]) & mask;
      w[p + h] ^= t;
      w[p] ^= t << (2 * h);
    }
  }
  // The four lanes of a quad hold the four dwords of a row's slab: exchange
  // them (4 x 4), so that a lane stores whole rows, 16 bytes each.
  const bool odd = d & 1, upper = d & 2;
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(odd ? w[j] : w[j + 1]), 0xB1, 0xF, 0xF, false);
    w[j] = odd ? y : w[j];
    w[j + 1] = odd ? w[j + 1] : y;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (j & 2) continue;
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(upper ? w[j] : w[j + 2]), 0x4E, 0xF, 0xF, false);
    w[j] = upper ? y : w[j];
    w[j + 2] = upper ? w[j + 2] : y;
  }
#pragma unroll
  for (int j = 0; j < 16; j += 4)
    if (k + j < A.k)  // K % 4 == 0
      *G(reinterpret_cast<v4i*>(A.ut + (slab * A.k + k + j + d) * kCodes)) =
          v4i{(int32_t)w[j], (int32_t)w[j + 1], (int32_t)w[j + 2], (int32_t)w[j + 3]};
}

// 2048 x 4096 x 14336, both gradients (150 MB moved): 31 us from memory, 4.9 TB/s.
__global__ __launch_bounds__(256) void prepare_kernel(const PrepArgs A) {
  const int wg = blockIdx.x;
  if (wg >= A.begin[2])
    prepare_weights(A, wg - A.begin[2]);
  else if (wg >= A.begin[1])
    prepare_xhat(A, wg - A.begin[1]);
  else
    prepare_dy(A, wg);
}

// ---------------------------------------------------------------------------
// The matrix products

struct GemmJob {
  const uint8_t* a;  // [slabs][ra] rows of 128 bytes, a_row and a_slab bytes apart
  const uint8_t* b;  // [slabs][rb] rows of 128 bytes, or 16 (two-bit weights)
  int64_t a_row, a_slab;
  int32_t ra, rb;    // C is [ra][rb]; rb % 4 == 0
  int32_t slabs;
  int32_t tiles_i, tiles_j;
  int32_t ksplit, kspw;  // parts of c and slabs per part
  int32_t cfg;           // tile size (kConfigs)
  int32_t codes;         // 1: b holds two-bit weights, c is half of the product's sum
  float* part;           // ksplit > 1: fp32 sums [ksplit][ra][rb]
  float* cf;             // fp32 output [ra][rb] (+ what is there), or nullptr
  int32_t accumulate;
  uint16_t* cb;          // bf16 output [ra][rb] = c / *scale (+ res)
  const float* scale;
  const uint16_t* res;
  // 1: the output is more than the L2 caches hold (32 MB), and is stored past
  // them: kept there it would push out the operands, and be written back at
  // the kernel's end (2048 x 4096 x 14336: 472 -> 437 us for both gradients)
  int32_t past_cache;
};

struct GemmArgs {
  GemmJob j[2];
  int32_t begin[3];  // first workgroup of each job (multiples of 8), of the bias sums
  // bias sums
  const float* dbp;
  int32_t dbp_rows, n;
  float* db;
  int32_t accumulate;
};

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

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");  // no LDS access moves across
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Eight weights (four dwords of two bf16 each) from two-bit codes: q holds
// pair a at bits 8 + 2a and 24 + 2a.  A byte select looks the high bytes of
// u / 2 up (-0.5, 0, 0.5: their low bytes are zero); shift, mask-or, select.
// The mask and the constant bytes are kept in registers (one scalar, one
// vector), where the mask-or is a single instruction.
struct Expand {
  uint32_t mask, zero;
  __device__ __forceinline__ Expand() : mask(0x03000300u), zero(0x000C000Cu) {
    asm("" : "+s"(mask));
    asm("" : "+v"(zero));
  }
  __device__ __forceinline__ v4i operator()(uint32_t q) const {
    v4i r;
#pragma unroll
    for (int a = 0; a < 4; ++a)
      r[a] = (int32_t)__builtin_amdgcn_perm(0u, 0x003F00BFu, ((q >> (2 * a)) & mask) | zero);
    return r;
  }
};

// Output of four columns of one row.
template <typename V, typename P>
__device__ __forceinline__ void put(V v, P* p, bool past_cache) {
  if (past_cache) {
    // fenced: the compiler would make one store of the two branches', a plain one
    asm volatile("" ::: "memory");
    __builtin_nontemporal_store(v, G(reinterpret_cast<V*>(p)));
    asm volatile("" ::: "memory");
  } else {
    *G(reinterpret_cast<V*>(p)) = v;
  }
}

__device__ __forceinline__ void put4(const GemmJob& J, int64_t o, v4f v, float scale) {
  if (J.cf) {
    if (J.accumulate) v += *G(reinterpret_cast<const v4f*>(J.cf + o));
    put(v, J.cf + o, J.past_cache);
    return;
  }
  v2i w;
  // c is half of the sum (Expand): doubling is exact
  w.x = (int32_t)pack_bf16x2(2.0f * v[0] / scale, 2.0f * v[1] / scale);
  w.y = (int32_t)pack_bf16x2(2.0f * v[2] / scale, 2.0f * v[3] / scale);
  if (J.res) {
    const v2i r = *G(reinterpret_cast<const v2i*>(J.res + o));
    w.x = (int32_t)add_bf16x2((uint32_t)w.x, (uint32_t)r.x);
    w.y = (int32_t)add_bf16x2((uint32_t)w.y, (uint32_t)r.y);
  }
  put(w, J.cb + o, J.past_cache);
}

// Bytes of one slab of both operands.
constexpr int stage_bytes(int ti, int tj, bool codes) { return ti * kRow + tj * (codes ? kCodes : kRow); }

// One tile of TI x TJ by WI x WJ waves.  Slabs of both operands go from
// global memory straight into a ring of NST buffers in LDS.  Chunk c (16
// bytes) of row r of a slab sits at chunk c ^ ((r / 2) & 7) of its 128-byte
// row, so that the 16 rows that LDS serves together lie in distinct banks.
template <int TI, int TJ, int WI, int WJ, int NST, bool CODES>
__device__ __forceinline__ void gemm_tile(const GemmJob& J, int ti, int tj, int kp, int8_t* smem) {
  constexpr int NW = WI * WJ;
  constexpr int FI = TI / WI / 32, FJ = TJ / WJ / 32;
  constexpr int kStage = stage_bytes(TI, TJ, CODES);
  constexpr int DA = TI / 8 / NW, DB = CODES ? 1 : TJ / 8 / NW;
  constexpr int CW = TJ / 64;  // CODES: DMA instructions that hold a slab's codes
  static_assert(DA * 8 * NW == TI && (CODES || DB * 8 * NW == TJ) && NW % CW == 0, "whole loads");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lr = lane & 31, lg = lane >> 5;
  const int i0 = ti * TI, j0 = tj * TJ;
  const int wi0 = (wave % WI) * (TI / WI), wj0 = (wave / WI) * (TJ / WJ);
  const int s0 = kp * J.kspw, nsl = min(J.slabs - s0, J.kspw);

  // Per lane the offsets within a slab, per wave the slab's address.
  uint32_t oa[DA], ob[DB];
  const int64_t step_a = J.a_slab, step_b = (int64_t)J.rb * (CODES ? kCodes : kRow);
  const uint8_t *pa = J.a + s0 * step_a + i0 * J.a_row, *pb = J.b + s0 * step_b;
#pragma unroll
  for (int i = 0; i < DA; ++i) {
    const int pos = (wave * DA + i) * 64 + lane, r = pos >> 3;
    oa[i] = (uint32_t)min(r, J.ra - 1 - i0) * (uint32_t)J.a_row + 16 * ((pos & 7) ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int i = 0; i < DB; ++i) {
    if constexpr (CODES) {  // waves past CW load the same codes again, so that all wait alike
      ob[i] = (uint32_t)min(j0 + (wave % CW) * 64 + lane, J.rb - 1) * kCodes;
    } else {
      const int pos = (wave * DB + i) * 64 + lane, r = pos >> 3;
      ob[i] = (uint32_t)min(j0 + r, J.rb - 1) * kRow + 16 * ((pos & 7) ^ ((r >> 1) & 7));
    }
  }
  // Load d (of DA + DB) of the next slab into the buffer st.
  constexpr int D = DA + DB;
  auto issue_one = [&](int d, int8_t* st) {
    if (d < DA)
      dma16(pa + oa[d], st + (wave * DA + d) * 1024);
    else
      dma16(pb + ob[d - DA], st + TI * kRow + (CODES ? wave % CW : wave * DB + d - DA) * 1024);
    if (d == D - 1) {
      pa += step_a;
      pb += step_b;
    }
  };

  v16f acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  const Expand expand;
  // Fragments of step ks of a slab: 16 c, eight a lane half.
  v4i fa[2][FI], fb[2][FJ], cj[FJ];
  const int8_t* sa = smem;  // the current slab's buffer
  auto load = [&](int ks, v4i (&a)[FI], v4i (&b)[FJ]) {
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const int r = wi0 + 32 * i + lr;
      a[i] = *reinterpret_cast<const v4i*>(sa + kRow * r + 16 * ((2 * ks + lg) ^ ((r >> 1) & 7)));
    }
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
      const int r = wj0 + 32 * j + lr;
      if constexpr (!CODES)
        b[j] = *reinterpret_cast<const v4i*>(sa + TI * kRow + kRow * r + 16 * ((2 * ks + lg) ^ ((r >> 1) & 7)));
      else if (ks == 0)
        b[j] = *reinterpret_cast<const v4i*>(sa + TI * kRow + kCodes * r);
    }
  };
  // Products of step ks; with ISSUE, a load of the slab that goes to `st`
  // between any two of them (all at once would hold up the products behind
  // them).
  auto multiply = [&](auto issue, int ks, const v4i (&a)[FI], const v4i (&b)[FJ], int8_t* st) {
    constexpr bool ISSUE = decltype(issue)::value;
    constexpr int P = FI * FJ;
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
      v4i w;
      if constexpr (CODES)
        w = expand((uint32_t)cj[j][ks] << (8 - 8 * lg));  // the lane half's eight c
      else
        w = b[j];
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        acc[i][j] = mfma_32x32x16(w, a[i], acc[i][j]);
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
  };

  constexpr int KS = kSlab / 16;
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
  // A slab: its first steps, then, when its last fragments are in registers
  // and every wave is there, its buffer is free.  The next slab's first
  // fragments are read ahead of the last products, and the buffer refilled
  // between them.
  auto slab = [&](auto issue, int s) {
    constexpr bool ISSUE = decltype(issue)::value;
    if constexpr (CODES) {
#pragma unroll
      for (int j = 0; j < FJ; ++j) cj[j] = fb[0][j];
    }
#pragma unroll
    for (int ks = 0; ks < KS - 1; ++ks) {
      load(ks + 1, fa[(ks + 1) & 1], fb[(ks + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);  // the reads go out ahead of this step's products
      multiply(std::false_type{}, ks, fa[ks & 1], fb[ks & 1], nullptr);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slab's LDS reads are done
    int8_t* st = smem + buf * kStage;
    if (ISSUE || s + 1 < nsl) {
      wait_vm<ISSUE ? (NST - 2) * D : 0>();
      barrier();
      buf = buf + 1 == NST ? 0 : buf + 1;
      sa = smem + buf * kStage;
      load(0, fa[0], fb[0]);
    }
    __builtin_amdgcn_sched_barrier(0);
    multiply(issue, KS - 1, fa[(KS - 1) & 1], fb[(KS - 1) & 1], st);
  };
  int s = 0;
  for (; s + NST < nsl; ++s) slab(std::true_type{}, s);
  for (; s < nsl; ++s) slab(std::false_type{}, s);

  // B is the matrix core's first operand: lane (lr, lg) holds, of each
  // subtile, row lr at columns 8 e + 4 lg .. + 3 in elements 4 e .. 4 e + 3
  // (rb % 4 == 0: such a run is whole or outside).  Stored like that, an
  // instruction would touch 32 rows; a pass through LDS, 32 rows of the wave's
  // columns at a time in a part of its own, makes it whole rows (the ring is
  // done with: its last loads have landed, and every wave is here).
  barrier();
  const float sc = !J.cf ? load_f32_vmem(J.scale) : 1.0f;
  constexpr int kPitch = 32 * FJ * 4 + 16;  // 16 bytes off: rows start at distinct banks
  static_assert(NW * 32 * kPitch <= NST * kStage, "the parts fit the ring");
  constexpr int LPR = 8 * FJ, RPI = 64 / LPR;  // lanes a row, rows an instruction
  int8_t* mine = smem + wave * 32 * kPitch;
#pragma unroll
  for (int i = 0; i < FI; ++i) {
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<v4f*>(mine + lr * kPitch + 4 * (32 * j + 8 * e + 4 * lg)) =
            v4f{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < 32 / RPI; ++q) {
      const int row = q * RPI + lane / LPR;
      const v4f v = *reinterpret_cast<const v4f*>(mine + row * kPitch + 16 * (lane % LPR));
      const int r = i0 + wi0 + 32 * i + row, c = j0 + wj0 + 4 * (lane % LPR);
      if (r >= J.ra || c >= J.rb) continue;
      const int64_t o = (int64_t)r * J.rb + c;
      if (J.ksplit > 1)
        *G(reinterpret_cast<v4f*>(J.part + (int64_t)kp * J.ra * J.rb + o)) = v;
      else
        put4(J, o, v, sc);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Workgroups go to the 8 XCDs round-robin and each has its own L2, so each XCD
// takes one contiguous share of a job's tiles, walked in groups of up to four
// tile rows so that neighbours in time share operands both ways.
__device__ __forceinline__ bool tile_of(int l, const GemmJob& J, int* ti, int* tj, int* kp) {
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

// The kernels: tiles of 64 x 64 and 128 x 128, whichever the plan takes for
// each product, by four waves (two workgroups a CU), and tiles of 256 x 256 by
// eight.  Slab rings are as deep as the LDS allows (two-bit slabs are smaller).
// 2048 x 4096 x 14336, both gradients: 416 us on average over 120 calls, 385 the
// shortest (466 and 413 on another MI355X), 1156 TFLOP/s, the matrix cores busy 60%
// of the cycles; 2048 x 6912 x 2560: 136 us, 126 the shortest.  What bounds them is
// the clock that the power of the products leaves: the same launch on zeros takes
// 319 us in place of 417, and the two of 4096 cubed 180 in place of 238, next to 92
// and 125 of one bf16 library product of that size.  Loads that always hit the
// caches gain 4% on dw and nothing on dx; tiles of 128 x 256, two workgroups a CU
// that do not wait for each other, gain nothing (dx of 4096 cubed 115 us against
// 112, of 2048 x 4096 x 14336 205 against 203).
constexpr int kDeep64 = 4, kDeep64c = 8, kDeep128 = 2, kDeep128c = 4, kDeep256 = 2, kDeep256c = 4;
constexpr int ring_bytes(int t, int deep, int deepc) {
  return std::max(deep * stage_bytes(t, t, false), deepc * stage_bytes(t, t, true));
}
constexpr size_t kLdsSmall = std::max(ring_bytes(64, kDeep64, kDeep64c), ring_bytes(128, kDeep128, kDeep128c));
constexpr size_t kLdsBig = ring_bytes(256, kDeep256, kDeep256c);
static_assert(2 * kLdsSmall <= 160 * 1024 && kLdsBig <= 160 * 1024, "LDS of a CU");

template <bool BIG>
__global__ __launch_bounds__(BIG ? 512 : 256, 2) void gemm_kernel(const GemmArgs A) {
  extern __shared__ __align__(16) int8_t smem[];
  const int wg = blockIdx.x;
  if (wg >= A.begin[2]) {  // bias sums: one column a thread, the slabs' sums in order
    const int c = (wg - A.begin[2]) * (BIG ? 512 : 256) + (int)threadIdx.x;
    if (c >= A.n) return;
    float s = 0.0f;
    for (int r = 0; r < A.dbp_rows; ++r) s += *G(A.dbp + (int64_t)r * A.n + c);
    *G(A.db + c) = A.accumulate ? *G(A.db + c) + s : s;
    return;
  }
  const int ji = wg >= A.begin[1] ? 1 : 0;
  const GemmJob& J = A.j[ji];
  int ti, tj, kp;
  if (!tile_of(wg - A.begin[ji], J, &ti, &tj, &kp)) return;
  if constexpr (BIG) {
    if (J.codes)
      gemm_tile<256, 256, 2, 4, kDeep256c, true>(J, ti, tj, kp, smem);
    else
      gemm_tile<256, 256, 2, 4, kDeep256, false>(J, ti, tj, kp, smem);
  } else if (J.cfg == 1) {
    if (J.codes)
      gemm_tile<128, 128, 2, 2, kDeep128c, true>(J, ti, tj, kp, smem);
    else
      gemm_tile<128, 128, 2, 2, kDeep128, false>(J, ti, tj, kp, smem);
  } else {
    if (J.codes)
      gemm_tile<64, 64, 2, 2, kDeep64c, true>(J, ti, tj, kp, smem);
    else
      gemm_tile<64, 64, 2, 2, kDeep64, false>(J, ti, tj, kp, smem);
  }
}

// Adds the parts of the split products, in order: four columns a thread.
__global__ __launch_bounds__(256) void gemm_finish_kernel(const GemmArgs A, int64_t first1, int64_t total) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= total) return;
  const GemmJob& J = A.j[id >= first1 ? 1 : 0];
  const int64_t o = 4 * (id - (id >= first1 ? first1 : 0)), slice = (int64_t)J.ra * J.rb;
  v4f v = *G(reinterpret_cast<const v4f*>(J.part + o));
  for (int p = 1; p < J.ksplit; ++p) v += *G(reinterpret_cast<const v4f*>(J.part + p * slice + o));
  put4(J, o, v, !J.cf ? load_f32_vmem(J.scale) : 1.0f);
}

// ---------------------------------------------------------------------------
// Small products, in one launch: a workgroup lays its operands out itself.
//
// Tiles of 64 x 64 by four waves of 32 x 32, c in steps of 128 (two slabs) from
// registers to one of two LDS buffers while the other multiplies.  Operands
// that several tiles share are laid out again by each, and a step waits for
// its loads: worth it while there are few steps next to a second launch and the
// trip of the operands through memory (both gradients of 16 x 480 x 960, whole
// calls: 8.7 us against 11.7).  At the border the plan's estimate is off by
// about 5%: 301 x 1001 x 1284, 8 steps, which it gives to this kernel, takes 16.8
// us here and 16.0 in two launches.

struct DirectArgs {
  int64_t m, n, k;
  const uint16_t* dy;
  const uint8_t* packed;
  int32_t tiled;
  const int8_t* q;
  const float* x_scale;
  float* db;
  int32_t tiles_k;    // tiles along K
  int32_t dw_begin;   // first workgroup of dw
  GemmJob dx, dw;     // their outputs
};

constexpr int kDirectA = 64 * kRow, kDirectB = 64 * kRow;  // bytes of a slab
constexpr int kDirectBuf = 2 * (kDirectA + kDirectB);

// Place of chunk c (16 bytes) of row r in a slab's image.
__device__ __forceinline__ int image(int r, int c) { return kRow * r + 16 * (c ^ ((r >> 1) & 7)); }

// Operand steps of dw: a lane takes 8 tokens x 4 columns of dy and of xhat;
// lanes 0-7 side by side a column's 64 tokens, waves 0 and 1 (2 and 3) the two
// slabs of the first (last) 32 columns.
struct DirectDw {
  const DirectArgs& A;
  int64_t i0, j0;
  bool sums;  // this tile also sums dy's columns
  v2i d[8];
  uint32_t c[8];
  float xs[8], sum[4];
  __device__ __forceinline__ DirectDw(const DirectArgs& a, int64_t i, int64_t j) : A(a), i0(i), j0(j) {
    sums = A.db && j0 == 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = 0.0f;
  }
  __device__ __forceinline__ int column() const {
    return 4 * (8 * ((int)threadIdx.x >> 7) + (((int)threadIdx.x >> 3) & 7));
  }
  __device__ __forceinline__ int slab() const { return ((int)threadIdx.x >> 6) & 1; }
  __device__ __forceinline__ void load(int64_t c0) {
    const int64_t m0 = c0 + 64 * slab() + 8 * (threadIdx.x & 7), n = i0 + column(), k = j0 + column();
    const int mv = (int)min((int64_t)8, A.m - m0);  // tokens that exist (may be <= 0)
    const int nv = (int)min((int64_t)4, A.n - n);
    const bool kv = k < A.k;  // K % 4 == 0
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // tokens that do not exist read the last one
      const int64_t m = min(m0 + i, A.m - 1);
      c[i] = *G(reinterpret_cast<const uint32_t*>(A.q + m * A.k + (kv ? k : 0)));
      xs[i] = *G(A.x_scale + m);
    }
    if (nv >= 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d[i] = *G(reinterpret_cast<const v2i_any*>(A.dy + min(m0 + i, A.m - 1) * A.n + n));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = v2i{0, 0};
#pragma unroll 1
      for (int e = 0; e < nv; ++e) {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *G(A.dy + min(m0 + i, A.m - 1) * A.n + n + e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i].x |= (int32_t)(e < 2 ? v[i] << (16 * (e & 1)) : 0u);
          d[i].y |= (int32_t)(e < 2 ? 0u : v[i] << (16 * (e & 1)));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= mv) d[i] = v2i{0, 0};
      if (i >= mv || !kv) c[i] = 0u;
    }
  }
  // Column j of the eight tokens' four bf16 values, as a 16-byte chunk.
  static __device__ __forceinline__ v4i column4(const v2i (&r)[8], int j) {
    v4i o;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      o[p] = (int32_t)__builtin_amdgcn_perm((uint32_t)r[2 * p + 1][j >> 1], (uint32_t)r[2 * p][j >> 1],
                                            (j & 1) ? 0x07060302u : 0x05040100u);
    return o;
  }
  __device__ __forceinline__ void store(int8_t* buf) {
    v2i x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const RestoreRow r = restore_row(xs[i]);
      x[i] = v2i{(int32_t)restore2(c[i], 0, r), (int32_t)restore2(c[i], 2, r)};
    }
    const int mi = threadIdx.x & 7, col = column();
    int8_t* at = buf + kDirectA * slab();
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<v4i*>(at + image(col + j, mi)) = column4(d, j);
    at = buf + 2 * kDirectA + kDirectB * slab();
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<v4i*>(at + image(col + j, mi)) = column4(x, j);
    if (sums) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = (uint32_t)d[i][e >> 1];
          sum[e] += __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
        }
    }
  }
  __device__ __forceinline__ void finish(int8_t* smem) {
    if (!sums) return;
    float* red = reinterpret_cast<float*>(smem);  // the buffers are done with
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float s = sum[e];
      s += __shfl_xor(s, 1);
      s += __shfl_xor(s, 2);
      s += __shfl_xor(s, 4);
      if ((threadIdx.x & 7) == e) red[64 * slab() + column() + e] = s;
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < 64 && i0 + t < A.n) {
      const float s = red[t] + red[64 + t];
      *G(A.db + i0 + t) = A.dw.accumulate ? *G(A.db + i0 + t) + s : s;
    }
  }
};

// Operand steps of dx: dy's rows as they are, four 16-byte chunks a thread;
// waves 2 and 3 transpose the weights, 16 rows n of one byte (four k) a lane.
struct DirectDx {
  const DirectArgs& A;
  int64_t i0, j0;
  v4i a[4];
  uint32_t w[4];
  __device__ __forceinline__ DirectDx(const DirectArgs& x, int64_t i, int64_t j) : A(x), i0(i), j0(j) {}
  __device__ __forceinline__ void load(int64_t c0) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t row = min(i0 + (tid >> 4) + 16 * q, A.m - 1), n = c0 + 8 * (tid & 15);
      const int nv = (int)min((int64_t)8, A.n - n);
      const uint16_t* p = A.dy + row * A.n + n;
      a[q] = v4i{0, 0, 0, 0};
      if (nv >= 8) {
        a[q] = *G(reinterpret_cast<const v4i_any*>(p));
      } else {
        uint64_t lo = 0, hi = 0;
#pragma unroll 1
        for (int e = 0; e < nv; ++e) {
          const uint64_t v = (uint64_t)*G(p + e) << (16 * (e & 3));
          lo |= e < 4 ? v : 0;
          hi |= e < 4 ? 0 : v;
        }
        a[q] = v4i{(int32_t)lo, (int32_t)(lo >> 32), (int32_t)hi, (int32_t)(hi >> 32)};
      }
    }
    if (tid < 128) return;
    // byte b of w[r] is row n0 + order(4 b + r): in the result the codes of
    // n = 2a and 2a + 1 then sit at bits 2a and 16 + 2a, as Expand takes them.
    // The 16 rows are a fixed stride apart in either layout (n0 % 16 == 0).
    const int64_t rb = A.k >> 2, n0 = c0 + 16 * ((tid - 128) >> 4);
    const int64_t o = min((j0 >> 2) + (tid & 15), rb - 1);
    const int last = (int)min((int64_t)15, A.n - 1 - n0);  // its rows that exist (may be < 0)
    const uint8_t* base = A.packed + (last < 0 ? 0 : A.tiled ? tiled_chunk_offset(n0, o & ~(int64_t)15, rb) + (o & 15) : n0 * rb + o);
    const uint32_t stride = A.tiled ? 16u : (uint32_t)rb;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint32_t v[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int p = 4 * b + r, row = p < 8 ? 2 * p : 2 * (p - 8) + 1;
        v[b] = *G(base + (uint32_t)max(0, min(row, last)) * stride);
        if (row > last) v[b] = 0x55u;  // rows past N: code 1, u = 0
      }
      w[r] = v[0] | (v[1] << 8) | (v[2] << 16) | (v[3] << 24);
    }
  }
  __device__ __forceinline__ void store(int8_t* buf) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = (tid >> 4) + 16 * q, c = tid & 15;
      *reinterpret_cast<v4i*>(buf + kDirectA * (c >> 3) + image(r, c & 7)) = a[q];
    }
    if (tid < 128) return;
    // 4 x 4 exchange of the two-bit fields of every byte
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t t = ((w[r] >> 4) ^ w[r + 2]) & 0x0F0F0F0Fu;
      w[r + 2] ^= t;
      w[r] ^= t << 4;
    }
#pragma unroll
    for (int r = 0; r < 4; r += 2) {
      const uint32_t t = ((w[r] >> 2) ^ w[r + 1]) & 0x33333333u;
      w[r + 1] ^= t;
      w[r] ^= t << 2;
    }
    const int d = (tid - 128) >> 4, k = 4 * (tid & 15);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint32_t*>(buf + 2 * kDirectA + kDirectB * (d >> 2) + kCodes * (k + j) + 4 * (d & 3)) = w[j];
  }
  __device__ __forceinline__ void finish(int8_t*) {}
};

template <bool CODES, typename Operands>
__device__ __forceinline__ void direct_tile(const DirectArgs& A, const GemmJob& J, Operands& op, int64_t c_len,
                                            int8_t* smem) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 31, lg = lane >> 5;
  const int wi0 = (wave & 1) * 32, wj0 = (wave >> 1) * 32;
  const Expand expand;
  v16f acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
  op.load(0);
  op.store(smem);
  __syncthreads();
  int at = 0;
  for (int64_t c0 = 0; c0 < c_len; c0 += kStep, at ^= 1) {
    const bool more = c0 + kStep < c_len;
    if (more) op.load(c0 + kStep);
    const int8_t* buf = smem + at * kDirectBuf;
    v4i fa[8], fb[8], cj[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int8_t* sa = buf + kDirectA * s;
      const int8_t* sb = buf + 2 * kDirectA + kDirectB * s;
      if constexpr (CODES) cj[s] = *reinterpret_cast<const v4i*>(sb + kCodes * (wj0 + lr));
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        fa[4 * s + ks] = *reinterpret_cast<const v4i*>(sa + image(wi0 + lr, 2 * ks + lg));
        if constexpr (!CODES) fb[4 * s + ks] = *reinterpret_cast<const v4i*>(sb + image(wj0 + lr, 2 * ks + lg));
      }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      v4i w;
      if constexpr (CODES)
        w = expand((uint32_t)cj[t >> 2][t & 3] << (8 - 8 * lg));
      else
        w = fb[t];
      acc = mfma_32x32x16(w, fa[t], acc);
    }
    if (more) op.store(smem + (at ^ 1) * kDirectBuf);
    __syncthreads();
  }
  op.finish(smem);
  const float sc = !J.cf ? load_f32_vmem(J.scale) : 1.0f;
  const int64_t r = op.i0 + wi0 + lr;
  if (r >= J.ra) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t c = op.j0 + wj0 + 8 * e + 4 * lg;
    if (c >= J.rb) continue;
    put4(J, r * J.rb + c, v4f{acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]}, sc);
  }
}

__global__ __launch_bounds__(256, 2) void direct_kernel(const DirectArgs A) {
  __shared__ __align__(16) int8_t smem[2 * kDirectBuf];
  const bool dw = (int)blockIdx.x >= A.dw_begin;
  const int t = dw ? (int)blockIdx.x - A.dw_begin : (int)blockIdx.x;
  const int64_t i0 = (int64_t)(t / A.tiles_k) * 64, j0 = (int64_t)(t % A.tiles_k) * 64;
  if (dw) {
    DirectDw op(A, i0, j0);
    direct_tile<false>(A, A.dw, op, A.m, smem);
  } else {
    DirectDx op(A, i0, j0);
    direct_tile<true>(A, A.dx, op, A.n, smem);
  }
}

// ---------------------------------------------------------------------------
constexpr int64_t kL2Bytes = int64_t(32) << 20;  // eight XCDs' L2

struct WsLayout {
  BackwardPlan plan;
  size_t dys, dyt, dbp, xt, ut, part[2], total;
};

WsLayout layout(int64_t m, int64_t n, int64_t k, bool dx, bool dw) {
  WsLayout L = {};
  const BackwardPlan p = L.plan = plan_backward(m, n, k, dx, dw);
  if (p.direct) return L;  // no workspace
  auto take = [&](size_t& off, bool want, int64_t bytes) {
    off = L.total;
    if (want) L.total = align256(L.total + (size_t)bytes);
  };
  take(L.dys, dx && !dy_as_is(n), slabs_of(n) * m * kRow);
  take(L.ut, dx, slabs_of(n) * k * kCodes);
  take(L.dyt, dw, slabs_of(m) * n * kRow);
  take(L.xt, dw, slabs_of(m) * k * kRow);
  take(L.dbp, dw, slabs_of(m) * n * 4);
  take(L.part[0], dx && p.ksplit[0] > 1, 4 * p.ksplit[0] * m * k);
  take(L.part[1], dw && p.ksplit[1] > 1, 4 * p.ksplit[1] * n * k);
  return L;
}

template <bool BIG>
hipError_t launch_gemm(const GemmArgs& a, int64_t wgs, hipStream_t s) {
  constexpr size_t lds = BIG ? kLdsBig : kLdsSmall;
  static_assert(lds > 64 * 1024, "the attribute is needed above 64 KB");
  static std::atomic<bool> done[kMaxDevices];  // once per device
  const int dev = current_device_index();
  if (!done[dev].load(std::memory_order_acquire)) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&gemm_kernel<BIG>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    done[dev].store(true, std::memory_order_release);
  }
  gemm_kernel<BIG><<<(unsigned)wgs, BIG ? 512 : 256, lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t backward_bytes(int64_t m, int64_t n, int64_t k, bool dx, bool dw) {
  return layout(m, n, k, dx, dw).total;
}

hipError_t launch_backward(const BackwardArgs& b, char* ws, size_t ws_bytes, hipStream_t s) {
  const bool dx = b.dx != nullptr, dw = b.dw != nullptr;
  const WsLayout L = layout(b.m, b.n, b.k, dx, dw);
  const BackwardPlan& p = L.plan;
  if (ws_bytes < L.total) return hipErrorInvalidValue;
  if (p.direct) {
    DirectArgs d = {};
    d.m = b.m;
    d.n = b.n;
    d.k = b.k;
    d.dy = b.dy;
    d.packed = b.packed;
    d.tiled = b.tiled ? 1 : 0;
    d.q = b.q;
    d.x_scale = b.x_scale;
    d.db = b.dbias;
    d.tiles_k = (int32_t)((b.k + 63) / 64);
    d.dx.ra = (int32_t)b.m;
    d.dw.ra = (int32_t)b.n;
    d.dx.rb = d.dw.rb = (int32_t)b.k;
    d.dx.cb = b.dx;
    d.dx.scale = b.w_scale;
    d.dx.res = b.residual;
    d.dw.cf = b.dw;
    d.dw.accumulate = b.accumulate ? 1 : 0;
    d.dw_begin = dx ? (int32_t)((b.m + 63) / 64) * d.tiles_k : 0;
    const int64_t wgs = d.dw_begin + (dw ? (b.n + 63) / 64 * d.tiles_k : 0);
    direct_kernel<<<(unsigned)wgs, 256, 0, s>>>(d);
    return hipGetLastError();
  }
  const int64_t ms = slabs_of(b.m), ns = slabs_of(b.n);

  PrepArgs pa = {};
  pa.m = b.m;
  pa.n = b.n;
  pa.k = b.k;
  pa.dy = b.dy;
  pa.dys = dx && !dy_as_is(b.n) ? reinterpret_cast<uint16_t*>(ws + L.dys) : nullptr;
  pa.dyt = dw ? reinterpret_cast<uint16_t*>(ws + L.dyt) : nullptr;
  pa.dbp = b.dbias ? reinterpret_cast<float*>(ws + L.dbp) : nullptr;
  pa.q = b.q;
  pa.x_scale = b.x_scale;
  pa.xt = reinterpret_cast<uint16_t*>(ws + L.xt);
  pa.packed = b.packed;
  pa.tiled = b.tiled ? 1 : 0;
  pa.ut = reinterpret_cast<uint8_t*>(ws + L.ut);
  int64_t wgs = pa.dys || dw ? ms * ((b.n + 255) / 256) : 0;
  pa.begin[0] = 0;
  pa.begin[1] = (int32_t)wgs;
  if (dw) wgs += ms * ((b.k + 255) / 256);
  pa.begin[2] = (int32_t)wgs;
  if (dx) wgs += ns * ((b.k + 1023) / 1024);
  prepare_kernel<<<(unsigned)wgs, 256, 0, s>>>(pa);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  GemmArgs g = {};
  const int64_t rows[2] = {b.m, b.n}, slabs[2] = {ns, ms};
  const bool want[2] = {dx, dw};
  const bool big = p.cfg[0] == 2;
  int64_t grid = 0, finish[2] = {0, 0};
  for (int o = 0; o < 2; ++o) {
    const int j = o == 0 ? p.order : 1 - p.order;  // 0: dx, 1: dw
    GemmJob& J = g.j[o];
    g.begin[o] = (int32_t)grid;
    if (!want[j]) continue;
    J.a = reinterpret_cast<const uint8_t*>(ws + (j ? L.dyt : L.dys));
    J.a_row = kRow;
    J.a_slab = rows[j] * kRow;
    if (j == 0 && dy_as_is(b.n)) {
      J.a = reinterpret_cast<const uint8_t*>(b.dy);
      J.a_row = 2 * b.n;
      J.a_slab = kRow;
    }
    J.b = reinterpret_cast<const uint8_t*>(ws + (j ? L.xt : L.ut));
    J.ra = (int32_t)rows[j];
    J.rb = (int32_t)b.k;
    J.slabs = (int32_t)slabs[j];
    J.tiles_i = (int32_t)((rows[j] + kConfigs[p.cfg[j]].ti - 1) / kConfigs[p.cfg[j]].ti);
    J.tiles_j = (int32_t)((b.k + kConfigs[p.cfg[j]].tj - 1) / kConfigs[p.cfg[j]].tj);
    J.ksplit = p.ksplit[j];
    J.kspw = p.kspw[j];
    J.cfg = p.cfg[j];
    J.codes = j == 0;
    J.part = reinterpret_cast<float*>(ws + L.part[j]);
    J.cf = j ? b.dw : nullptr;
    J.accumulate = b.accumulate ? 1 : 0;
    J.cb = j ? nullptr : b.dx;
    J.scale = b.w_scale;
    J.res = j ? nullptr : b.residual;
    J.past_cache = rows[j] * b.k * (j ? 4 : 2) > kL2Bytes ? 1 : 0;
    if (J.ksplit > 1) finish[o] = rows[j] * (b.k / 4);
    grid += round_up((int64_t)J.tiles_i * J.tiles_j * J.ksplit, 8);
  }
  g.begin[2] = (int32_t)grid;
  if (b.dbias) {
    g.dbp = pa.dbp;
    g.dbp_rows = (int32_t)ms;
    g.n = (int32_t)b.n;
    g.db = b.dbias;
    g.accumulate = b.accumulate ? 1 : 0;
    const int threads = big ? 512 : 256;
    grid += (b.n + threads - 1) / threads;
  }
  e = big ? launch_gemm<true>(g, grid, s) : launch_gemm<false>(g, grid, s);
  const int64_t total = finish[0] + finish[1];
  if (e != hipSuccess || total == 0) return e;
  gemm_finish_kernel<<<(unsigned)((total + 255) / 256), 256, 0, s>>>(g, finish[0], total);
  return hipGetLastError();
}

}  // namespace bl
