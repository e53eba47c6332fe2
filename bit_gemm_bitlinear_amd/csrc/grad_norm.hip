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

constexpr int kTensors = 100;        // a launch (its arguments are at most 4 KB)
constexpr int64_t kChunk = 1 << 14;  // elements of one tensor that a workgroup takes at a time
constexpr int kMaxParts = 2048;      // partial sums, workgroups of a launch

struct NormTensor {
  const void* g;
  void* out;
  int64_t numel;
  int32_t chunk_begin;  // first chunk of the launch
  int32_t flags;        // 1: bf16, 2: pointers 16-byte aligned
};

struct GradNormArgs {
  NormTensor t[kTensors];
  int32_t count, chunks;
  double* parts;  // this launch's partial sums (norm pass)
  const double* all;
  int32_t nall;
  float max_norm;
  float* norm;  // or nullptr
};
static_assert(sizeof(GradNormArgs) <= 4096, "kernel arguments");

__device__ __forceinline__ int tensor_of(const GradNormArgs& A, int chunk) {
  int lo = 0, hi = A.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (A.t[mid].chunk_begin <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double s, double* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__device__ __forceinline__ float element(const void* p, int64_t i, bool bf16) {
  return bf16 ? bf16_to_f32(*G(reinterpret_cast<const uint16_t*>(p) + i)) : *G(reinterpret_cast<const float*>(p) + i);
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const GradNormArgs A) {
  __shared__ double red[4];
  double s = 0.0;
  for (int c = blockIdx.x; c < A.chunks; c += gridDim.x) {
    const NormTensor& T = A.t[tensor_of(A, c)];
    const int64_t b = (int64_t)(c - T.chunk_begin) * kChunk, e = min(b + kChunk, T.numel);
    for (int64_t i = b + threadIdx.x; i < e; i += 256) {
      const double v = element(T.g, i, T.flags & 1);
      s = fma(v, v, s);
    }
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) *G(A.parts + blockIdx.x) = s;
}

__device__ __forceinline__ double total_of(const GradNormArgs& A, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < A.nall; i += 256) s += *G(A.all + i);
  return block_sum(s, red);
}

__global__ __launch_bounds__(256) void grad_norm_finish_kernel(const GradNormArgs A) {
  __shared__ double red[4];
  const double s = total_of(A, red);
  if (threadIdx.x == 0) *G(A.norm) = (float)sqrt(s);
}

__global__ __launch_bounds__(256) void grad_clip_kernel(const GradNormArgs A) {
  __shared__ double red[4];
  const double norm = sqrt(total_of(A, red)), r = (double)A.max_norm / (norm + 1e-6);
  const float f = r >= 1.0 ? 1.0f : (float)r;  // NaN stays NaN
  if (A.norm && blockIdx.x == 0 && threadIdx.x == 0) *G(A.norm) = (float)norm;
  for (int c = blockIdx.x; c < A.chunks; c += gridDim.x) {
    const NormTensor& T = A.t[tensor_of(A, c)];
    if (f == 1.0f && T.g == T.out) continue;  // in place, and nothing to change
    const int64_t b = (int64_t)(c - T.chunk_begin) * kChunk, e = min(b + kChunk, T.numel);
    for (int64_t i = b + threadIdx.x; i < e; i += 256) {
      const float v = element(T.g, i, T.flags & 1) * f;
      if (T.flags & 1)
        *G(reinterpret_cast<uint16_t*>(T.out) + i) = f32_to_bf16(v);
      else
        *G(reinterpret_cast<float*>(T.out) + i) = v;
    }
  }
}

int64_t chunks_of(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

}  // namespace

// Every launch of tensors leaves up to kMaxParts partial sums.
size_t grad_norm_bytes(int32_t count, const int64_t* numel) {
  size_t parts = 0;
  for (int32_t i = 0; i < count; i += kTensors) {
    int64_t chunks = 0;
    for (int32_t j = i; j < std::min(count, i + kTensors); ++j) chunks += chunks_of(numel[j]);
    parts += (size_t)std::min<int64_t>(chunks, kMaxParts);
  }
  return align256(8 * std::max<size_t>(parts, 1));
}

hipError_t launch_grad_norm(int32_t count, const Gradient* t, bool clip, float max_norm, float* norm, char* ws,
                            hipStream_t s) {
  GradNormArgs a = {};
  a.all = reinterpret_cast<const double*>(ws);
  a.max_norm = max_norm;
  for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
    int32_t parts = 0;
    for (int32_t i = 0; i < count; i += kTensors) {
      int64_t chunks = 0;
      a.count = 0;
      for (int32_t j = i; j < std::min(count, i + kTensors); ++j) {
        if (t[j].numel == 0) continue;
        NormTensor& T = a.t[a.count++];
        T.g = t[j].g;
        T.out = t[j].out;
        T.numel = t[j].numel;
        T.chunk_begin = (int32_t)chunks;
        const uintptr_t bits = reinterpret_cast<uintptr_t>(T.g) | reinterpret_cast<uintptr_t>(clip ? T.out : T.g);
        T.flags = (t[j].bf16 ? 1 : 0) | ((bits & 15) ? 0 : 2);
        chunks += chunks_of(T.numel);
      }
      if (chunks == 0) continue;
      a.chunks = (int32_t)chunks;
      const unsigned grid = (unsigned)std::min<int64_t>(chunks, kMaxParts);
      if (pass == 0) {
        a.parts = reinterpret_cast<double*>(ws) + parts;
        parts += (int32_t)grid;
        grad_norm_kernel<<<grid, 256, 0, s>>>(a);
      } else {
        grad_clip_kernel<<<grid, 256, 0, s>>>(a);
        a.norm = nullptr;  // written by the first of them
      }
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    a.nall = pass == 0 ? parts : a.nall;
    a.norm = norm;
    if ((pass == 0 && !clip) || parts + a.nall == 0) {
      // no clipping pass, or no element at all
      grad_norm_finish_kernel<<<1, 256, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  return hipSuccess;
}

}  // namespace bl
