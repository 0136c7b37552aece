// Backward pass of the combine: out[t] = x[t] + sum over kept choices of gate * y.
//
//   dgates[t, c] = sum_j dout[t, j] y[slot, j]      (0 for a dropped choice)
//   dy[slot]     = gate dout[t]
// (the residual's part of dx is dout itself.)
//
// Bound: HBM, one read of dout and of the kept rows of y, one write of dy.  One wave a token: its slots
// first, then the token's row of dout once for up to kB choices at a time, with the rows of all of
// them in flight: 2, 4 or 8, the least that holds top_k (T 16384, d 2048, top-6 with dy, 643 MB: 151, 148
// and 145 us with 2, 4 and 8; T 64, top-2 without: 3.5, 4.0 and 4.8).  Products of bf16 are exact in fp32
// and summed in fp32, lane by lane and then over the wave, in a fixed order.
#include "router_rows.h"

namespace moe {

namespace {

struct CombineBackArgs {
  const void* dout;
  const float* gates;  // with dy
  const int32_t* slot_of;
  const void* y;  // with dgates
  float* dgates;  // may be NULL
  void* dy;       // may be NULL
  int64_t T;
  int d, k;
  uint32_t rows;  // of y and dy; a slot past them is a dropped choice's, as -1 is
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// V columns of a row, widened: 8 bf16 or 4 fp32 in 16 bytes, or one fp32.  Stores of 16 bytes go past
// the caches, as moe_combine's do (T 16384, d 2048, top-6: 150 -> 148 us).
template <typename T, int V>
struct Piece;
template <>
struct Piece<bf16_t, 8> {
  uint4 v;
  static constexpr int kBytes = 16;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) { v = buffer_load16(r, off); }
  __device__ __forceinline__ void widen(float (&o)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(char* p, const float (&o)[8]) {
    const u32x4 w = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                     pack_bf16x2(o[6], o[7])};
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
  }
};
template <>
struct Piece<float, 4> {
  uint4 v;
  static constexpr int kBytes = 16;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) { v = buffer_load16(r, off); }
  __device__ __forceinline__ void widen(float (&o)[4]) const {
    o[0] = __uint_as_float(v.x), o[1] = __uint_as_float(v.y);
    o[2] = __uint_as_float(v.z), o[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ void store(char* p, const float (&o)[4]) {
    const f32x4 w = {o[0], o[1], o[2], o[3]};
    __builtin_nontemporal_store(w, reinterpret_cast<f32x4*>(p));
  }
};
template <>
struct Piece<float, 1> {
  float v;
  static constexpr int kBytes = 4;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) { v = buffer_load_f32(r, off); }
  __device__ __forceinline__ void widen(float (&o)[1]) const { o[0] = v; }
  static __device__ __forceinline__ void store(char* p, const float (&o)[1]) {
    *reinterpret_cast<float*>(p) = o[0];
  }
};

__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum<16>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

template <typename T, int V, bool DY, int kB>
__global__ __launch_bounds__(256) void k_combine_back(const CombineBackArgs a) {
  using P = Piece<T, V>;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const uint32_t row_bytes = (uint32_t)a.d * (uint32_t)sizeof(T);
  const __amdgpu_buffer_rsrc_t dr = buffer_rsrc((const char*)a.dout + t * row_bytes, row_bytes);
  for (int c0 = 0; c0 < a.k; c0 += kB) {
    int slot[kB];
    float gate[kB], acc[kB];
    __amdgpu_buffer_rsrc_t yr[kB];
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      slot[j] = c0 + j < a.k ? a.slot_of[t * a.k + c0 + j] : -1;
      if ((uint32_t)slot[j] >= a.rows) slot[j] = -1;
      gate[j] = DY && slot[j] >= 0 ? a.gates[t * a.k + c0 + j] : 0.0f;
      acc[j] = 0.0f;
      // the row of a dropped choice has no bytes: it reads as zeros
      const bool read = a.dgates && slot[j] >= 0;
      yr[j] = buffer_rsrc((const char*)a.y + (int64_t)(read ? slot[j] : 0) * row_bytes,
                          read ? row_bytes : 0u);
    }
    for (uint32_t off = lane * P::kBytes; off < row_bytes; off += 64 * P::kBytes) {
      P dp, yp[kB];
      dp.load(dr, off);
#pragma unroll
      for (int j = 0; j < kB; ++j) yp[j].load(yr[j], off);
      float dv[V];
      dp.widen(dv);
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        float yv[V];
        yp[j].widen(yv);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[j] = fmaf(dv[i], yv[i], acc[j]);
        if (DY && slot[j] >= 0) {
          float o[V];
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = gate[j] * dv[i];
          P::store((char*)a.dy + (int64_t)slot[j] * row_bytes + off, o);
        }
      }
    }
    if (a.dgates) {
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const float s = wave_sum(acc[j]);
        // a dropped choice: zero whatever dout holds
        if (lane == 0 && c0 + j < a.k) a.dgates[t * a.k + c0 + j] = slot[j] >= 0 ? s : 0.0f;
      }
    }
  }
}

template <typename T, int V>
hipError_t launch(const CombineBackArgs& a, hipStream_t st) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, st, a);
    return hipGetLastError();
  };
  if (a.k <= 2) return a.dy ? go(k_combine_back<T, V, true, 2>) : go(k_combine_back<T, V, false, 2>);
  if (a.k <= 4) return a.dy ? go(k_combine_back<T, V, true, 4>) : go(k_combine_back<T, V, false, 4>);
  return a.dy ? go(k_combine_back<T, V, true, 8>) : go(k_combine_back<T, V, false, 8>);
}

}  // namespace

hipError_t launch_combine_backward(const moe_shape& s, const void* dout, const float* gates,
                                   const int32_t* slot_of, const void* y, int64_t rows,
                                   float* dgates, void* dy, hipStream_t st) {
  const size_t size = s.dtype == MOE_BF16 ? 2 : 4, row = (size_t)s.d_model * size;
  constexpr int64_t kTokens = 1 << 25;  // a launch: 64 threads each, and 2^32 are too many
  for (int64_t t = 0; t < s.T; t += kTokens) {
    const int64_t n = s.T - t < kTokens ? s.T - t : kTokens;
    const CombineBackArgs a{(const char*)dout + t * row, gates ? gates + t * s.top_k : nullptr,
                            slot_of + t * s.top_k, y, dgates ? dgates + t * s.top_k : nullptr, dy, n,
                            s.d_model, s.top_k, (uint32_t)(rows < INT32_MAX ? rows : INT32_MAX)};
    const uintptr_t all = (uintptr_t)dout | (uintptr_t)y | (uintptr_t)dy;
    hipError_t err;
    if (s.dtype == MOE_BF16)
      err = launch<bf16_t, 8>(a, st);
    else if (s.d_model % 4 == 0 && all % 16 == 0)
      err = launch<float, 4>(a, st);
    else
      err = launch<float, 1>(a, st);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
