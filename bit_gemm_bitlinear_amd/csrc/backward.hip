// Gradients of BitLinear from its 8-bit activation checkpoint.
//
//   dx[m][k] = bf16( sum_n dy[m][n] * u[n][k] / w_scale )
//   dw[n][k] = sum_m dy[m][n] * xhat[m][k],  xhat = bf16(q / x_scale)
//   db[n]    = sum_m dy[m][n]
//
// u in {-1, 0, 1} and xhat are bf16 values, so every product is exact in the
// bf16 matrix cores' fp32 sums.  Both are matrix products C[i][j] = sum_c
// A[i][c] B[j][c] of operands whose summed index c is contiguous; what is
// stored the other way round is transposed into the workspace first (dy and
// the restored activations for dw, the expanded weights for dx), with c padded
// by zeros to whole slabs.
#include "../../include/bitlinear_layer.h"
#include "common.hpp"
#include "internal.hpp"
#include "layer_internal.hpp"

#include <atomic>

namespace bl {

namespace {

constexpr int kSlab = 64;  // c per slab: 128 bytes of a bf16 row

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v16f mfma_32x32x16(v4i a, v4i b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a),
                                                 __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// ---- operands laid out with the summed index contiguous ----

// 64 x 64 tiles of src [rows][cols] (bf16) to dst [cols][ldd], dst columns
// past `rows` zeroed.
// KIND 0: bf16 as it is.  1: int8 codes q restored to bf16(q / x_scale[row]).
// 2: packed ternary weights [rows][cols / 4] as bf16 u; `tiled`: their layout.
template <int KIND>
__global__ __launch_bounds__(256) void transpose_kernel(const void* __restrict__ src,
                                                        const float* __restrict__ x_scale,
                                                        int64_t rows, int64_t cols, int tiled,
                                                        uint16_t* __restrict__ dst, int64_t ldd) {
  __shared__ uint16_t t[64][66];
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll 4
  for (int i = ty; i < 64; i += 4) {
    const int64_t r = r0 + i, c = c0 + tx;
    uint16_t v = 0;
    if (r < rows && c < cols) {
      if constexpr (KIND == 0) {
        v = *G(static_cast<const uint16_t*>(src) + r * cols + c);
      } else if constexpr (KIND == 1) {
        v = f32_to_bf16((float)*G(static_cast<const int8_t*>(src) + r * cols + c) / *G(x_scale + r));
      } else {
        const int64_t rb = cols / 4, o = c >> 2;
        const int64_t off = tiled ? tiled_chunk_offset(r, o & ~(int64_t)15, rb) + (o & 15) : r * rb + o;
        const uint32_t code = (*G(static_cast<const uint8_t*>(src) + off) >> (2 * (c & 3))) & 3u;
        v = f32_to_bf16((float)((int)code - 1));
      }
    }
    t[i][tx] = v;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = ty; i < 64; i += 4) {
    const int64_t c = c0 + i;
    if (c < cols) *G(dst + c * ldd + r0 + tx) = t[tx][i];
  }
}

// Rows of dy [m][n] copied to [m][ldd], zero-padded: only where n % 8 != 0
// (the matrix product reads 16-byte aligned rows).
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ src, int64_t m,
                                                       int64_t n, uint16_t* __restrict__ dst,
                                                       int64_t ldd) {
  for (int64_t r = blockIdx.y; r < m; r += gridDim.y) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c < ldd) *G(dst + r * ldd + c) = c < n ? *G(src + r * n + c) : (uint16_t)0;
  }
}

// db: one wave per row of the transposed dy.
__global__ __launch_bounds__(256) void row_sum_kernel(const uint16_t* __restrict__ a, int64_t rows,
                                                      int64_t ld, float* __restrict__ out,
                                                      int accumulate) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= rows) return;
  float s = 0.0f;
  for (int64_t c = 8 * lane; c < ld; c += 512) {
    const v4i v = *G(reinterpret_cast<const v4i*>(a + r * ld + c));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s += __uint_as_float((uint32_t)v[i] << 16) + __uint_as_float((uint32_t)v[i] & 0xFFFF0000u);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) out[r] = accumulate ? out[r] + s : s;
}

// ---- the matrix product ----

struct GemmArgs {
  const uint16_t* a;  // [ra][lda]
  const uint16_t* b;  // [rb][ldb]
  int64_t lda, ldb;
  int32_t ra, rb;      // rows of A and B: C is [ra][rb]
  int32_t ca;          // columns of A that hold data (a multiple of 8; chunks past them
                       // are read from the row's last one and meet zeros in B)
  int32_t slabs;       // of kSlab
  int32_t tiles_i, tiles_j;
  // output
  float* cf;           // fp32 [ra][rb], or nullptr
  int32_t accumulate;  // cf: add to what is there
  uint16_t* cb;        // bf16 [ra][rb] of c / *scale (+ res), or nullptr
  const float* scale;
  const uint16_t* res;
};

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

__device__ __forceinline__ void dma16(const void* src, int8_t* lds_dst) {
  __builtin_amdgcn_global_load_lds((const BL_GLOBAL void*)src,
                                   (__attribute__((address_space(3))) void*)lds_dst, 16, 0, 0);
}

// Tile TI x TJ with WI x WJ waves.  Slabs of both operands go from global
// memory straight into LDS, two buffers: slab s + 1 is in flight while slab s
// is multiplied.  Chunk c (16 bytes) of row r of a slab sits at chunk
// c ^ ((r / 2) & 7) of its 128-byte row, so that the 16 rows that LDS serves
// together lie in distinct banks.
template <int TI, int TJ, int WI, int WJ>
__global__ __launch_bounds__(64 * WI * WJ) void gemm_kernel(const GemmArgs A) {
  constexpr int NT = 64 * WI * WJ;
  constexpr int FI = TI / WI / 32, FJ = TJ / WJ / 32;
  constexpr int kStage = (TI + TJ) * 128;
  constexpr int DA = TI * 8 / NT, DB = TJ * 8 / NT;
  extern __shared__ __align__(16) int8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 31, lg = lane >> 5;
  const int ti = (int)(blockIdx.x % (unsigned)A.tiles_i), tj = (int)(blockIdx.x / (unsigned)A.tiles_i);
  const int i0 = ti * TI, j0 = tj * TJ;
  const int wi0 = (wave % WI) * (TI / WI), wj0 = (wave / WI) * (TJ / WJ);

  const uint16_t* pa[DA];
  int ca[DA];
  const uint16_t* pb[DB];
#pragma unroll
  for (int i = 0; i < DA; ++i) {
    const int pos = (wave * DA + i) * 64 + lane, r = pos >> 3;
    ca[i] = 8 * ((pos & 7) ^ ((r >> 1) & 7));
    pa[i] = A.a + (int64_t)min(i0 + r, A.ra - 1) * A.lda;
  }
#pragma unroll
  for (int i = 0; i < DB; ++i) {
    const int pos = (wave * DB + i) * 64 + lane, r = pos >> 3;
    pb[i] = A.b + (int64_t)min(j0 + r, A.rb - 1) * A.ldb + 8 * ((pos & 7) ^ ((r >> 1) & 7));
  }
  auto issue = [&](int s, int8_t* st) {
#pragma unroll
    for (int i = 0; i < DA; ++i)
      dma16(pa[i] + min(s * kSlab + ca[i], A.ca - 8), st + (wave * DA + i) * 1024);
#pragma unroll
    for (int i = 0; i < DB; ++i)
      dma16(pb[i] + s * kSlab, st + TI * 128 + (wave * DB + i) * 1024);
  };

  v16f acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  issue(0, smem);
  for (int s = 0; s < A.slabs; ++s) {
    wait_vm<0>();
    __builtin_amdgcn_s_barrier();
    if (s + 1 < A.slabs) issue(s + 1, smem + ((s + 1) & 1) * kStage);
    const int8_t* sa = smem + (s & 1) * kStage;
    const int8_t* sb = sa + TI * 128;
#pragma unroll
    for (int ks = 0; ks < kSlab / 16; ++ks) {
      v4i fa[FI], fb[FJ];
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        const int r = wi0 + 32 * i + lr;
        fa[i] = *reinterpret_cast<const v4i*>(sa + 128 * r + 16 * ((2 * ks + lg) ^ ((r >> 1) & 7)));
      }
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int r = wj0 + 32 * j + lr;
        fb[j] = *reinterpret_cast<const v4i*>(sb + 128 * r + 16 * ((2 * ks + lg) ^ ((r >> 1) & 7)));
      }
#pragma unroll
      for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = mfma_32x32x16(fa[i], fb[j], acc[i][j]);
    }
  }

  // lane (lr, lg) holds rows 8 (e / 4) + 4 lg + e % 4 of column lr of each subtile
  const float sc = A.cb ? load_f32_vmem(A.scale) : 1.0f;
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int r = i0 + wi0 + 32 * i + 8 * (e >> 2) + 4 * lg + (e & 3);
      if (r >= A.ra) continue;
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int c = j0 + wj0 + 32 * j + lr;
        if (c >= A.rb) continue;
        const int64_t o = (int64_t)r * A.rb + c;
        if (A.cf) {
          *G(A.cf + o) = A.accumulate ? *G(A.cf + o) + acc[i][j][e] : acc[i][j][e];
        } else {
          uint16_t v = f32_to_bf16(acc[i][j][e] / sc);
          if (A.res) v = add_bf16(v, *G(A.res + o));
          *G(A.cb + o) = v;
        }
      }
    }
}

template <int TI, int TJ, int WI, int WJ>
hipError_t launch_gemm(GemmArgs a, hipStream_t s) {
  constexpr size_t lds = 2 * (TI + TJ) * 128;
  if (lds > 64 * 1024) {  // the attribute is needed above 64 KB; once per device
    static std::atomic<bool> done[kMaxDevices];
    const int dev = current_device_index();
    if (!done[dev].load(std::memory_order_acquire)) {
      const hipError_t e = hipFuncSetAttribute(
          reinterpret_cast<const void*>(&gemm_kernel<TI, TJ, WI, WJ>),
          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
      done[dev].store(true, std::memory_order_release);
    }
  }
  a.tiles_i = (a.ra + TI - 1) / TI;
  a.tiles_j = (a.rb + TJ - 1) / TJ;
  const int64_t tiles = (int64_t)a.tiles_i * a.tiles_j;
  gemm_kernel<TI, TJ, WI, WJ><<<(unsigned)tiles, 64 * WI * WJ, lds, s>>>(a);
  return hipGetLastError();
}

hipError_t gemm(const GemmArgs& a, hipStream_t s) {
  const int64_t big = (int64_t)((a.ra + 255) / 256) * ((a.rb + 255) / 256);
  if (big >= 256) return launch_gemm<256, 256, 2, 4>(a, s);
  return launch_gemm<128, 128, 2, 2>(a, s);
}

size_t bf16_bytes(int64_t rows, int64_t ld) { return align256((size_t)rows * (size_t)ld * 2); }

dim3 tiles64(int64_t rows, int64_t cols) {
  return dim3((unsigned)((cols + 63) / 64), (unsigned)((rows + 63) / 64));
}

}  // namespace

size_t backward_input_bytes(int64_t m, int64_t n, int64_t k) {
  const int64_t np = round_up(n, kSlab);
  return bf16_bytes(k, np) + (n % 8 ? bf16_bytes(m, np) : 0);
}

hipError_t launch_backward_input(int64_t m, int64_t n, int64_t k, const uint16_t* dy,
                                 const uint8_t* packed, bool tiled, const float* w_scale,
                                 const uint16_t* residual, uint16_t* dx, char* ws, hipStream_t s) {
  const int64_t np = round_up(n, kSlab);
  uint16_t* ut = reinterpret_cast<uint16_t*>(ws);
  transpose_kernel<2><<<tiles64(n, k), 256, 0, s>>>(packed, nullptr, n, k, tiled ? 1 : 0, ut, np);
  GemmArgs g = {};
  g.a = dy;
  g.lda = n;
  g.ca = (int32_t)n;
  if (n % 8) {
    uint16_t* p = reinterpret_cast<uint16_t*>(ws + bf16_bytes(k, np));
    pad_rows_kernel<<<dim3((unsigned)((np + 255) / 256), (unsigned)(m < 65535 ? m : 65535)), 256, 0, s>>>(
        dy, m, n, p, np);
    g.a = p;
    g.lda = np;
    g.ca = (int32_t)np;
  }
  g.b = ut;
  g.ldb = np;
  g.ra = (int32_t)m;
  g.rb = (int32_t)k;
  g.slabs = (int32_t)(np / kSlab);
  g.cb = dx;
  g.scale = w_scale;
  g.res = residual;
  return gemm(g, s);
}

size_t backward_weight_bytes(int64_t m, int64_t n, int64_t k) {
  const int64_t mp = round_up(m, kSlab);
  return bf16_bytes(n, mp) + bf16_bytes(k, mp);
}

hipError_t launch_backward_weight(int64_t m, int64_t n, int64_t k, const uint16_t* dy,
                                  const int8_t* q, const float* x_scale, float* dw, float* dbias,
                                  bool accumulate, char* ws, hipStream_t s) {
  const int64_t mp = round_up(m, kSlab);
  uint16_t* dyt = reinterpret_cast<uint16_t*>(ws);
  uint16_t* xt = reinterpret_cast<uint16_t*>(ws + bf16_bytes(n, mp));
  transpose_kernel<0><<<tiles64(m, n), 256, 0, s>>>(dy, nullptr, m, n, 0, dyt, mp);
  transpose_kernel<1><<<tiles64(m, k), 256, 0, s>>>(q, x_scale, m, k, 0, xt, mp);
  if (dbias)
    row_sum_kernel<<<(unsigned)((n + 3) / 4), 256, 0, s>>>(dyt, n, mp, dbias, accumulate ? 1 : 0);
  GemmArgs g = {};
  g.a = dyt;
  g.lda = mp;
  g.ca = (int32_t)mp;
  g.b = xt;
  g.ldb = mp;
  g.ra = (int32_t)n;
  g.rb = (int32_t)k;
  g.slabs = (int32_t)(mp / kSlab);
  g.cf = dw;
  g.accumulate = accumulate ? 1 : 0;
  return gemm(g, s);
}

}  // namespace bl
