// Rows of router logits in registers: how the balance loss and the router's backward pass hold
// one token's E <= 256 logits (not part of the C interface).
//
// LPT lanes (at most one 16-lane DPP row) hold one token, NV values each, so a wave takes
// 64 / LPT tokens at a time and every reduction over the experts is at most four DPP moves:
// VEC (E a multiple of 4): value 4 q + c of lane l is expert 4 (q LPT + l) + c, 16-byte loads;
// otherwise value i of lane l is expert i LPT + l, 4-byte loads.
#pragma once

#include "moe_internal.h"

namespace moe {

// Reductions over LPT = 1 .. 16 neighbouring lanes, the result in every one of them: partners 1
// and 2 lanes apart are quad permutations; once the four lanes of a quad agree, mirroring half a
// row and then a whole row of 16 meets the other quads.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp32<CTRL>(__float_as_uint(v)));
}
template <int LPT>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (LPT >= 2) v += dpp_f32<0xB1>(v);
  if constexpr (LPT >= 4) v += dpp_f32<0x4E>(v);
  if constexpr (LPT >= 8) v += dpp_f32<0x141>(v);
  if constexpr (LPT >= 16) v += dpp_f32<0x140>(v);
  return v;
}
template <int LPT>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (LPT >= 2) v = fmaxf(v, dpp_f32<0xB1>(v));
  if constexpr (LPT >= 4) v = fmaxf(v, dpp_f32<0x4E>(v));
  if constexpr (LPT >= 8) v = fmaxf(v, dpp_f32<0x141>(v));
  if constexpr (LPT >= 16) v = fmaxf(v, dpp_f32<0x140>(v));
  return v;
}

// e^x for x <= 0 (or NaN): 2^t with t = x log2(e) in two parts, so the product's rounding does
// not reach the result (relative error a few 2^-24 instead of |x| 2^-24).
__device__ __forceinline__ float exp_nonpositive(float x) {
  const float kHi = 1.44269502162933349609375f, kLo = 1.92596299e-8f, kLn2 = 0.693147182f;
  const float t = x * kHi;
  const float r = fmaf(x, kHi, -t) + x * kLo;  // what t lost, |r| <= 2^-23 |t|
  const float v = __builtin_amdgcn_exp2f(t);
  return x < -104.0f ? 0.0f : fmaf(v, r * kLn2, v);
}

template <int LPT_, int NV_, bool VEC_>
struct RouterRow {
  static constexpr int LPT = LPT_, NV = NV_;
  static constexpr bool VEC = VEC_;
  static constexpr int TPW = 64 / LPT;  // tokens a wave holds
  // expert of value i of lane l (of LPT); past E for padding
  static __device__ __forceinline__ int expert(int l, int i) {
    return VEC ? 4 * ((i / 4) * LPT + l) + i % 4 : i * LPT + l;
  }
  static __device__ __forceinline__ void load(const float* __restrict__ row, int E, int l,
                                              float pad, float (&v)[NV]) {
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) {
        const int e = 4 * (q * LPT + l);
        float4 f = make_float4(pad, pad, pad, pad);
        if (e < E) f = *reinterpret_cast<const float4*>(row + e);
        v[4 * q] = f.x;
        v[4 * q + 1] = f.y;
        v[4 * q + 2] = f.z;
        v[4 * q + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = i * LPT + l < E ? row[i * LPT + l] : pad;
    }
  }
  static __device__ __forceinline__ void store(float* __restrict__ row, int E, int l,
                                               const float (&v)[NV]) {
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) {
        const int e = 4 * (q * LPT + l);
        if (e < E)
          *reinterpret_cast<float4*>(row + e) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * LPT + l < E) row[i * LPT + l] = v[i];
    }
  }
  // logits -> softmax probabilities in place, fp32 (the padding's are 0).  A row whose logits are
  // all -inf sums to 0 and has probabilities 0.  The maximum leaves NaN out (the padding is -inf, so
  // it is -inf for a row of nothing but NaN, too); the exponentials do not, and the sum carries it
  // to the whole row.
  static __device__ __forceinline__ void softmax(float (&v)[NV]) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, v[i]);
    m = row_max<LPT>(m);
    m = m == -INFINITY ? 0.0f : m;  // -inf - 0 is -inf, where -inf - -inf would be NaN
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = exp_nonpositive(v[i] - m);
      s += v[i];
    }
    s = row_sum<LPT>(s);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;  // in any other row the maximum adds 1
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] *= inv;
  }
};

// Calls f(RouterRow<...>{}) with the narrowest row that holds E experts; vec: E is a multiple
// of 4 and the arrays are 16-byte aligned.
template <typename F>
auto with_router_row(int E, bool vec, F f) {
  if (vec) {
    if (E <= 4) return f(RouterRow<1, 4, true>{});
    if (E <= 8) return f(RouterRow<2, 4, true>{});
    if (E <= 16) return f(RouterRow<4, 4, true>{});
    if (E <= 32) return f(RouterRow<8, 4, true>{});
    if (E <= 64) return f(RouterRow<16, 4, true>{});
    if (E <= 128) return f(RouterRow<16, 8, true>{});
    return f(RouterRow<16, 16, true>{});
  }
  if (E <= 16) return f(RouterRow<16, 1, false>{});
  if (E <= 32) return f(RouterRow<16, 2, false>{});
  if (E <= 64) return f(RouterRow<16, 4, false>{});
  if (E <= 128) return f(RouterRow<16, 8, false>{});
  return f(RouterRow<16, 16, false>{});
}

}  // namespace moe
