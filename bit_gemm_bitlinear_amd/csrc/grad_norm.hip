// The norm of many gradients together, and the gradients clipped to it.
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = g * c
//
// Squares and sums are fp64 (the square of an fp32 value is exact there, and no
// sum of them overflows; one fused step a value, which memory hides).  Two passes
// over the gradients, as the factor needs the whole sum: the first leaves one
// partial sum a workgroup, the second adds them up again in every workgroup, in
// one order, so that the result does not depend on timing.  Tensors go by value
// in a launch's arguments, kTensors at a time.
#include "../../include/bitlinear_ffn.h"
#include "common.hpp"
#include "internal.hpp"
#include "layer_internal.hpp"

#include <algorithm>

namespace bl {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kTensors = 120;           // a launch (its arguments are at most 4 KB)
constexpr int kMaxParts = 2048;         // workgroups, and so partial sums, of a launch
// Elements of one tensor that a workgroup takes at a time: as many, or as few as give
// each workgroup two chunks (45 tensors of 13.8 MB: chunks down to 2K 12.3 us, to 8K
// 11.7, to 16K 11.8; 27 of 33 MB 22.7, 20.0 and 19.9).
constexpr int64_t kLongChunk = 1 << 15;
constexpr int64_t kShortChunk = 1 << 13;

struct NormTensor {
  const void* g;
  void* out;
  int64_t numel;
  int32_t first;  // its first chunk of the launch
  int32_t flags;  // 1: bf16, 2: g and out lie alike in 16-byte pieces, from element flags >> 2 on
};

struct GradNormArgs {
  NormTensor t[kTensors];
  int32_t count, chunks;
  int32_t chunk;  // elements
  float max_norm;
  double* parts;      // this launch's partial sums (norm pass)
  const double* all;  // every launch's
  int32_t nall;
  float* norm;  // or nullptr
};
static_assert(sizeof(GradNormArgs) <= 4096, "kernel arguments");

// The tensor of a chunk: each lane looks at two of them, in one round trip.
__device__ __forceinline__ int tensor_of(const GradNormArgs& A, int chunk) {
  const int lane = threadIdx.x & 63;
  const int a = lane < A.count ? A.t[lane].first : INT32_MAX;
  const int b = 64 + lane < A.count ? A.t[64 + lane].first : INT32_MAX;
  return __builtin_popcountll(__ballot(a <= chunk)) + __builtin_popcountll(__ballot(b <= chunk)) - 1;
}
static_assert(kTensors <= 128, "two a lane");

__device__ __forceinline__ double block_sum(double s, double* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// Calls body(first element, 16-byte piece) for the whole 16-byte pieces of chunk c of
// a tensor, up to D in flight, and one(i) for the elements before and after them (for
// all where g and out lie differently).  N: elements of a piece.  A tensor's pieces
// begin at element `head`, and so do its chunks but the first, which takes what is
// before (218 million elements, nine views of one buffer from odd elements on,
// clipped: element by element fp32 804 us and bf16 656, so 527 and 265).
template <int N, typename Load, typename Body, typename One>
__device__ __forceinline__ void pieces(const NormTensor& T, int64_t c, int64_t chunk, const Load& load,
                                       const Body& body, const One& one) {
  constexpr int D = 8;
  const int head = T.flags >> 2;
  const int64_t e = min((c + 1) * chunk + head, T.numel);
  int64_t b = c ? c * chunk + head : 0;
  if (T.flags & 2) {
    if (c == 0) {
      b = min((int64_t)head, e);
      if ((int)threadIdx.x < b) one(threadIdx.x);
    }
    for (int64_t i = b + N * threadIdx.x; i + N <= e; i += D * N * 256) {
      v4i v[D];
#pragma unroll
      for (int u = 0; u < D; ++u)
        if (i + u * N * 256 + N <= e) v[u] = load(i + u * N * 256);
#pragma unroll
      for (int u = 0; u < D; ++u)
        if (i + u * N * 256 + N <= e) body(i + u * N * 256, v[u]);
    }
    b = e - (e - b) % N;  // (of a last chunk with nothing in it: e or more)
  }
  for (int64_t j = b + threadIdx.x; j < e; j += 256) one(j);
}

// Squares and sum in fp64 of the 4 fp32 or 8 bf16 values of a piece.
__device__ __forceinline__ void add_squares(v4i v, bool bf16, double (&s)[4]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t w = (uint32_t)v[d];
    if (bf16) {
      const double lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
      s[d] = fma(lo, lo, s[d]);
      s[d] = fma(hi, hi, s[d]);
    } else {
      const double x = __uint_as_float(w);
      s[d] = fma(x, x, s[d]);
    }
  }
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const GradNormArgs A) {
  __shared__ double red[4];
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  for (int c = blockIdx.x; c < A.chunks; c += gridDim.x) {
    const NormTensor& T = A.t[tensor_of(A, c)];
    if (T.flags & 1) {
      const uint16_t* g = static_cast<const uint16_t*>(T.g);
      pieces<8>(T, c - T.first, A.chunk, [&](int64_t i) { return *G(reinterpret_cast<const v4i*>(g + i)); },
                [&](int64_t, v4i v) { add_squares(v, true, s); },
                [&](int64_t i) {
                  const double x = bf16_to_f32(*G(g + i));
                  s[0] = fma(x, x, s[0]);
                });
    } else {
      const float* g = static_cast<const float*>(T.g);
      pieces<4>(T, c - T.first, A.chunk, [&](int64_t i) { return *G(reinterpret_cast<const v4i*>(g + i)); },
                [&](int64_t, v4i v) { add_squares(v, false, s); },
                [&](int64_t i) {
                  const double x = *G(g + i);
                  s[0] = fma(x, x, s[0]);
                });
    }
  }
  const double sum = block_sum((s[0] + s[1]) + (s[2] + s[3]), red);
  if (threadIdx.x == 0) *G(A.parts + blockIdx.x) = sum;
}

__device__ __forceinline__ double total_of(const GradNormArgs& A, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < A.nall; i += 8 * 256) {
    double v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i + u * 256 < A.nall ? *G(A.all + i + u * 256) : 0.0;
#pragma unroll
    for (int u = 0; u < 8; ++u) s += v[u];
  }
  return block_sum(s, red);
}

__global__ __launch_bounds__(256) void grad_norm_finish_kernel(const GradNormArgs A) {
  __shared__ double red[4];
  const double s = total_of(A, red);
  if (threadIdx.x == 0) *G(A.norm) = (float)sqrt(s);
}

// Chunks from the last one on: the ones that the norm's pass read last are those
// that the last-level cache still holds.  The clipped values are stored past the
// caches (872 MB of fp32 in place, over and over: this pass 313 -> 322 us, 5.4 TB/s,
// the norm's 187 -> 145, 6.0 TB/s).
__global__ __launch_bounds__(256) void grad_clip_kernel(const GradNormArgs A) {
  __shared__ double red[4];
  const double norm = sqrt(total_of(A, red)), r = (double)A.max_norm / (norm + 1e-6);
  const float f = r >= 1.0 ? 1.0f : (float)r;  // NaN stays NaN
  if (A.norm && blockIdx.x == 0 && threadIdx.x == 0) *G(A.norm) = (float)norm;
  for (int c = A.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const NormTensor& T = A.t[tensor_of(A, c)];
    if (f == 1.0f && T.g == T.out) continue;  // in place, and nothing to change
    if (T.flags & 1) {
      const uint16_t* g = static_cast<const uint16_t*>(T.g);
      uint16_t* out = static_cast<uint16_t*>(T.out);
      pieces<8>(T, c - T.first, A.chunk, [&](int64_t i) { return *G(reinterpret_cast<const v4i*>(g + i)); },
                [&](int64_t i, v4i v) {
#pragma unroll
                  for (int d = 0; d < 4; ++d) {
                    const uint32_t w = (uint32_t)v[d];
                    v[d] = (int32_t)pack_bf16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
                  }
                  __builtin_nontemporal_store(v, G(reinterpret_cast<v4i*>(out + i)));
                },
                [&](int64_t i) { *G(out + i) = f32_to_bf16(bf16_to_f32(*G(g + i)) * f); });
    } else {
      const float* g = static_cast<const float*>(T.g);
      float* out = static_cast<float*>(T.out);
      pieces<4>(T, c - T.first, A.chunk, [&](int64_t i) { return *G(reinterpret_cast<const v4i*>(g + i)); },
                [&](int64_t i, v4i v) {
                  __builtin_nontemporal_store(__builtin_bit_cast(v4f, v) * f, G(reinterpret_cast<v4f*>(out + i)));
                },
                [&](int64_t i) { *G(out + i) = *G(g + i) * f; });
    }
  }
}

// The tensors [begin, end) of one launch, and their chunks.
struct Group {
  int32_t begin, end;
  int64_t chunk, chunks;
  int32_t parts() const { return (int32_t)std::min<int64_t>(chunks, kMaxParts); }
};

template <typename Numel>
Group group_at(int32_t begin, int32_t count, const Numel& numel) {
  Group g = {begin, std::min(count, begin + kTensors), kLongChunk, 0};
  for (; g.chunk >= kShortChunk; g.chunk /= 2) {
    g.chunks = 0;
    for (int32_t i = g.begin; i < g.end; ++i) g.chunks += (numel(i) + g.chunk - 1) / g.chunk;
    if (g.chunks >= 2 * kMaxParts || g.chunk == kShortChunk) break;
  }
  return g;
}

}  // namespace

size_t grad_norm_bytes(int32_t count, const int64_t* numel) {
  size_t parts = 0;
  for (int32_t i = 0; i < count; i += kTensors)
    parts += (size_t)group_at(i, count, [&](int32_t j) { return numel[j]; }).parts();
  return align256(8 * std::max<size_t>(parts, 1));
}

hipError_t launch_grad_norm(int32_t count, const Gradient* t, bool clip, float max_norm, float* norm, char* ws,
                            hipStream_t s) {
  GradNormArgs a = {};
  a.all = reinterpret_cast<const double*>(ws);
  a.max_norm = max_norm;
  const int32_t groups = (count + kTensors - 1) / kTensors;
  auto fill = [&](int32_t gi) {
    const Group g = group_at(gi * kTensors, count, [&](int32_t j) { return t[j].numel; });
    a.count = 0;
    a.chunk = (int32_t)g.chunk;
    a.chunks = (int32_t)g.chunks;
    int64_t first = 0;
    for (int32_t j = g.begin; j < g.end; ++j) {
      if (t[j].numel == 0) continue;
      const uintptr_t at = reinterpret_cast<uintptr_t>(t[j].g) & 15;
      const bool alike = !clip || at == (reinterpret_cast<uintptr_t>(t[j].out) & 15);
      const int32_t head = (int32_t)((16 - at) & 15) / (t[j].bf16 ? 2 : 4);
      a.t[a.count++] = NormTensor{t[j].g, t[j].out, t[j].numel, (int32_t)first,
                                  (t[j].bf16 ? 1 : 0) | (alike ? 2 | head << 2 : 0)};
      first += (t[j].numel + g.chunk - 1) / g.chunk;
    }
    return (unsigned)g.parts();
  };
  for (int32_t gi = 0; gi < groups; ++gi) {
    const unsigned grid = fill(gi);
    if (grid == 0) continue;  // no element
    a.parts = reinterpret_cast<double*>(ws) + a.nall;
    grad_norm_kernel<<<grid, 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.nall += (int32_t)grid;
  }
  a.norm = norm;
  if (clip && a.nall) {
    for (int32_t gi = groups - 1; gi >= 0; --gi) {  // the last tensors first (see grad_clip_kernel)
      const unsigned grid = fill(gi);
      if (grid == 0) continue;
      grad_clip_kernel<<<grid, 256, 0, s>>>(a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      a.norm = nullptr;  // written by the first of them
    }
    return hipSuccess;
  }
  grad_norm_finish_kernel<<<1, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bl
