// Operands of the routers' fp64 matrix instructions: 8 columns of a token or of an expert, loaded
// as they are stored and widened exactly to fp64 (not part of the C interface).
#pragma once

#include "moe_internal.h"

namespace moe {

// 8 bf16 (one 16-byte word) widened exactly to fp64
__device__ __forceinline__ void widen_bf16x8(uint4 q, double* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (double)__uint_as_float(w[i] << 16);
    v[2 * i + 1] = (double)__uint_as_float(w[i] & 0xFFFF0000u);
  }
}

typedef double f64x4_t __attribute__((ext_vector_type(4)));

template <typename TIn>
struct Chunk8;
// The loads go through buffer resources over the whole matrix: a guarded-off chunk reads zeros
// from an out-of-range offset instead of sitting in a branch, so the compiler can count the
// loads in flight and wait only for the ones it needs (a predicated load made it wait for all).
template <>
struct Chunk8<bf16_t> {  // 8 bf16 columns as one 16-byte load (d % 8 == 0 for bf16)
  uint4 v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t m, bool ok, int64_t row, int c,
                                       int d) {
    v = buffer_load16(m, ok && c * 8 < d ? (uint32_t)((row * d + (int64_t)c * 8) * 2) : kBufferOOR);
  }
  __device__ __forceinline__ void widen(double* o) const { widen_bf16x8(v, o); }
};
template <>
struct Chunk8<float> {  // 8 fp32 columns, each guarded (any d)
  float v[8];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t m, bool ok, int64_t row, int c,
                                       int d) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int col = c * 8 + u;
      v[u] = buffer_load_f32(m, ok && col < d ? (uint32_t)((row * d + col) * 4) : kBufferOOR);
    }
  }
  __device__ __forceinline__ void widen(double* o) const {
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] = v[u];
  }
};

}  // namespace moe
