// AdamW over many tensors at once, moments in fp32 or in 8 bits.
//
//   g' = grad_scale g
//   m  = beta1 m + (1 - beta1) g',   v = beta2 v + (1 - beta2) g'^2
//   p  = p - lr wd p - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
// m and v are fp32 numbers formed by the operations as written, each rounded (no fused ones), so that
// the 8-bit codes below are the same wherever they are computed; p takes the unquantised m and v.
//
// 8 bits: blocks of 256 consecutive elements of a tensor share one fp32 step for m and one for
// r = sqrt(v).  A code c stands for c |c| step (c = -127 .. 127) and for r = c^2 step (c = 0 .. 255);
// step = max |x| / c_max^2, c = the root of |x| / step rounded to nearest.  Squares, because the
// elements of a block differ by orders of magnitude: 2 / c apart relatively, down to 1 / c_max^2 of
// the largest.  r and not v, because r divides: its relative error is the update's.  An r that is not
// zero keeps a code of 1 at least.  Rounding to nearest: of a v that hardly moves (beta2 0.999) the
// steps of one pass are below half a code, so codes move only as the block's largest does and by
// large gradients, which still holds r within 6.5 % of fp32's on average over 4000 steps of Gaussian
// gradients whose size varies by e^(+-1) within a block; rounding at random, unbiased, adds its noise
// every step and holds it within 8 %.
//
// Bound: memory, 28 bytes an element for fp32 moments and gradients, 14 to 18 for 8 bits.  The tensors'
// addresses go along as kernel arguments, 48 to a launch; a block takes 1024 elements of one tensor, a
// thread 4 neighbours, so that a wave has exactly the 256 that share a step.
#include <math.h>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kTensors = 48;    // a launch
constexpr int kChunk = 1024;    // elements a block (4096 and 2048: 1326 and 1317 us against 1269 for 268
                                // million elements, 13.2 and 12.3 against 11.7 for 4.2 million)
constexpr int64_t kMaxBlocks = 1 << 23;  // a launch: 2^32 threads are too many
// From this many bytes on a pass, more than the last-level cache holds, 32-bit moments and what goes with
// them are loaded past the caches (1185 us against 1269 for 268 million elements, but 13.1 against 11.7
// where all of it stays in the cache from step to step).
constexpr int64_t kStreamBytes = (int64_t)256 << 20;
constexpr int kQuantBlock = 256;
static_assert(kChunk == 4 * 256, "a block's threads take 4 elements each");

struct AdamRec {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_steps;
  float* v_steps;
  bf16_t* copy;
  int64_t n;
  float wd;
  int vec;  // every array lies where 4 elements load at once
};
struct AdamArgs {
  AdamRec rec[kTensors];
  int32_t start[kTensors];  // first block of each tensor
  int32_t count;
  float lr, beta1, beta2, eps, grad_scale, rate, inv_root;
  double log_beta1, log_beta2;
  const float* dynamic;
};

struct Rates {
  float lr, grad_scale, rate, inv_root;
};

// The 4 elements of a lane, as loaded.
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <bool STREAM>
__device__ __forceinline__ void load4(const float* p, int64_t i, int64_t n, bool whole, float (&o)[4]) {
  if (whole) {
    const f32x4* at = reinterpret_cast<const f32x4*>(p + i);
    const f32x4 f = STREAM ? __builtin_nontemporal_load(at) : *at;
    o[0] = f[0], o[1] = f[1], o[2] = f[2], o[3] = f[3];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = i + j < n ? p[i + j] : 0.0f;
  }
}
template <bool STREAM>
__device__ __forceinline__ void load4(const bf16_t* p, int64_t i, int64_t n, bool whole, float (&o)[4]) {
  if (whole) {
    const uint64_t* at = reinterpret_cast<const uint64_t*>(p + i);
    const uint64_t f = STREAM ? __builtin_nontemporal_load(at) : *at;
    const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32);
    o[0] = __uint_as_float(lo << 16), o[1] = __uint_as_float(lo & 0xFFFF0000u);
    o[2] = __uint_as_float(hi << 16), o[3] = __uint_as_float(hi & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = i + j < n ? bf16_to_f32(p[i + j]) : 0.0f;
  }
}
// Stores go past the caches: nothing of a step is read again before the next one (moments of 37.8
// million elements 90 -> 63 us, the step on them 128 -> 124).
__device__ __forceinline__ void store4(float* p, int64_t i, int64_t n, bool whole,
                                       const float (&o)[4]) {
  if (whole) {
    const f32x4 w = {o[0], o[1], o[2], o[3]};
    __builtin_nontemporal_store(w, reinterpret_cast<f32x4*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = o[j];
  }
}
__device__ __forceinline__ void store4(bf16_t* p, int64_t i, int64_t n, bool whole,
                                       const float (&o)[4]) {
  const uint32_t a = pack_bf16x2(o[0], o[1]), b = pack_bf16x2(o[2], o[3]);
  if (whole) {
    __builtin_nontemporal_store((uint64_t)b << 32 | a, reinterpret_cast<uint64_t*>(p + i));
  } else {
    const bf16_t w[4] = {(bf16_t)a, (bf16_t)(a >> 16), (bf16_t)b, (bf16_t)(b >> 16)};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = w[j];
  }
}
// 4 codes in a dword, the first lowest
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int64_t n, bool whole) {
  if (whole) return *reinterpret_cast<const uint32_t*>(p + i);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) w |= (uint32_t)p[i + j] << (8 * j);
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, bool whole, uint32_t w) {
  if (whole) {
    __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = (uint8_t)(w >> (8 * j));
  }
}
__device__ __forceinline__ void decode_m(uint32_t w, float step, float (&o)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float c = (float)((int)(w << (24 - 8 * j)) >> 24);
    o[j] = c * fabsf(c) * step;  // the square is exact
  }
}
__device__ __forceinline__ void decode_v(uint32_t w, float step, float (&o)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float c = (float)((w >> (8 * j)) & 0xFFu), r = c * c * step;
    o[j] = r * r;
  }
}

// The largest of the wave's |x|, as their bit patterns order them: NaN above infinity above all else.
template <bool SIGNED>
__device__ __forceinline__ float wave_absmax(const float (&x)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u = SIGNED ? __float_as_uint(x[j]) & 0x7FFFFFFFu : __float_as_uint(x[j]);
    m = u > m ? u : m;
  }
  auto take = [&](uint32_t o) { m = o > m ? o : m; };
  take(dpp32<0xB1>(m));
  take(dpp32<0x4E>(m));
  take(dpp32<0x141>(m));
  take(dpp32<0x140>(m));
  const uint32_t a = __builtin_amdgcn_readlane(m, 0), b = __builtin_amdgcn_readlane(m, 16);
  const uint32_t c = __builtin_amdgcn_readlane(m, 32), d = __builtin_amdgcn_readlane(m, 48);
  const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
  return __uint_as_float(ab > cd ? ab : cd);
}
// The code of x under `step`, by the definition; a block whose step is not finite has no value left that
// is: codes 0 (or 1).
template <int TOP>
__device__ __forceinline__ int encode(float x, float step) {
  const float y = step > 0.0f ? fabsf(x) / step : 0.0f;
  const float c = floorf(sqrtf(y) + 0.5f);
  const int code = c >= 0.0f ? (int)fminf(c, (float)TOP) : 0;
  if (TOP == 255) return x > 0.0f && code < 1 ? 1 : code;
  return x < 0.0f ? -code : code;
}
// The codes of a lane's four values; exact(j) gives value j as the definition has it, x[j] may be a step
// of fp32 off.  Away from the borders between codes the hardware's reciprocal and root are near enough:
// x, the reciprocal and the product put |x| / step 2.5 steps off, its root 1.25 and one of its own,
// 2.25 2^-23 of at most 255.5 or 2^-13.8, and the sums with 1/2 and the definition's own roundings less
// than 2^-14 more.  A lane with a value within 2^-12 of a border (12 waves in 100 have one) does its
// values over, and so do all where the step is too small or large for its reciprocal, or no number.
template <int TOP, typename Exact>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], Exact exact, float step) {
  const float inv = __builtin_amdgcn_rcpf(step);
  float edge = 0.0f;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float f = __builtin_amdgcn_sqrtf(fabsf(x[j]) * inv) + 0.5f;
    edge = fmaxf(edge, fabsf(__builtin_amdgcn_fractf(f) - 0.5f));
    const uint32_t c = (uint32_t)f, bits = __float_as_uint(x[j]);
    if (TOP == 255) {  // x >= 0; not 0 where x is not
      const uint32_t least = bits < 1u ? bits : 1u;
      w |= (c < least ? least : c > 255u ? 255u : c) << (8 * j);
    } else {
      const uint32_t sign = (uint32_t)((int)bits >> 31);
      w |= ((((c > 127u ? 127u : c) ^ sign) - sign) & 0xFFu) << (8 * j);
    }
  }
  if (edge > 0.5f - 0x1p-12f || !(step > 0x1p-80f && step < 0x1p100f)) {
    w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= ((uint32_t)encode<TOP>(exact(j), step) & 0xFFu) << (8 * j);
  }
  return w;
}

// m and v of one element, each operation rounded
__device__ __forceinline__ void moments(float g, float beta1, float beta2, float& m, float& v) {
#pragma clang fp contract(off)
  const float keep_m = m * beta1, new_m = g * (1.0f - beta1);
  m = keep_m + new_m;
  const float sq = g * g;
  const float keep_v = v * beta2, new_v = sq * (1.0f - beta2);
  v = keep_v + new_v;
}

__device__ __forceinline__ int tensor_of(const int32_t* start, int count, int block) {
  const int lane = threadIdx.x & 63;
  const bool before = lane < count && start[lane < count ? lane : 0] <= block;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(before)) - 1);
}

template <typename P, typename G, bool Q8, bool STREAM>
__global__ __launch_bounds__(256) void k_adamw(const AdamArgs a) {
  const int ti = tensor_of(a.start, a.count, (int)blockIdx.x);
  const AdamRec& r = a.rec[ti];
  const int64_t n = r.n, base = (int64_t)((int)blockIdx.x - a.start[ti]) * kChunk;
  Rates c{a.lr, a.grad_scale, a.rate, a.inv_root};
  if (a.dynamic) {
    if (a.dynamic[3] != 0.0f) return;
    c.lr = a.dynamic[0];
    c.grad_scale = a.dynamic[1];
    const double t = fmax((double)a.dynamic[2], 1.0);
    c.rate = (float)((double)c.lr / -expm1(t * a.log_beta1));
    c.inv_root = (float)(1.0 / sqrt(-expm1(t * a.log_beta2)));
  }
  const float lr_wd = c.lr * r.wd;
  P* p = (P*)r.p;
  const G* g = (const G*)r.g;
  bf16_t* copy = r.copy;
  const bool whole = r.vec && base + kChunk <= n;
  const int64_t i = base + (int64_t)threadIdx.x * 4;
  if (!whole && base + (threadIdx.x & ~63) * 4 >= n) return;  // waves leave together
  float pv[4], gv[4], mv[4], vv[4];
  load4<STREAM>(p, i, n, whole, pv);
  load4<STREAM>(g, i, n, whole, gv);
  const int64_t qb = i / kQuantBlock;
  if constexpr (Q8) {
    decode_m(load_codes((const uint8_t*)r.m, i, n, whole), r.m_steps[qb], mv);
    decode_v(load_codes((const uint8_t*)r.v, i, n, whole), r.v_steps[qb], vv);
  } else {
    load4<STREAM>((const float*)r.m, i, n, whole, mv);
    load4<STREAM>((const float*)r.v, i, n, whole, vv);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) moments(gv[j] * c.grad_scale, a.beta1, a.beta2, mv[j], vv[j]);
  float rv[4];
  if constexpr (Q8) {
    // The kernel of 8 bits is short of instructions, not of bytes (122 an element with every root and
    // quotient in full: 139 us for 37.8 million elements): roots and the quotient to a step of fp32,
    // except roots of denormal numbers, which the instruction takes for zeros.
    uint32_t least = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = __float_as_uint(vv[j]) - 1u;  // 0 is fine
      least = u < least ? u : least;
      rv[j] = __builtin_amdgcn_sqrtf(vv[j]);
    }
    if (least < 0x007FFFFFu)
#pragma unroll
      for (int j = 0; j < 4; ++j) rv[j] = sqrtf(vv[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q = fmaf(-lr_wd, pv[j], pv[j]);
      pv[j] = fmaf(-c.rate * mv[j], __builtin_amdgcn_rcpf(fmaf(rv[j], c.inv_root, a.eps)), q);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q = fmaf(-lr_wd, pv[j], pv[j]);
      pv[j] = q - c.rate * mv[j] / fmaf(sqrtf(vv[j]), c.inv_root, a.eps);
    }
  }
  store4(p, i, n, whole, pv);
  if (copy) store4(copy, i, n, whole, pv);
  if constexpr (Q8) {
    // elements past the tensor's end are zeros; the largest root is the largest v's
    const float ms = wave_absmax<true>(mv) / 16129.0f, vs = sqrtf(wave_absmax<false>(vv)) / 65025.0f;
    const uint32_t mc = encode4<127>(mv, [&](int j) { return mv[j]; }, ms);
    const uint32_t vc = encode4<255>(rv, [&](int j) { return sqrtf(vv[j]); }, vs);
    store_codes((uint8_t*)r.m, i, n, whole, mc);
    store_codes((uint8_t*)r.v, i, n, whole, vc);
    if ((threadIdx.x & 63) == 0) {
      r.m_steps[qb] = ms;
      r.v_steps[qb] = vs;
    }
  } else {
    store4((float*)r.m, i, n, whole, mv);
    store4((float*)r.v, i, n, whole, vv);
  }
}

struct MomentRec {
  const void* m;
  const void* v;
  const float* m_steps;
  const float* v_steps;
  float* m_out;
  float* v_out;
  int64_t n;
  int vec;
};
struct MomentArgs {
  MomentRec rec[kTensors];
  int32_t start[kTensors];
  int32_t count;
};

template <bool Q8>
__global__ __launch_bounds__(256) void k_adamw_moments(const MomentArgs a) {
  const int ti = tensor_of(a.start, a.count, (int)blockIdx.x);
  const MomentRec& r = a.rec[ti];
  const int64_t n = r.n, base = (int64_t)((int)blockIdx.x - a.start[ti]) * kChunk;
  const bool whole = r.vec && base + kChunk <= n;
  const int64_t i = base + (int64_t)threadIdx.x * 4;
  if (i >= n) return;
  float mv[4], vv[4];
  if constexpr (Q8) {
    decode_m(load_codes((const uint8_t*)r.m, i, n, whole), r.m_steps[i / kQuantBlock], mv);
    decode_v(load_codes((const uint8_t*)r.v, i, n, whole), r.v_steps[i / kQuantBlock], vv);
  } else {
    load4<false>((const float*)r.m, i, n, whole, mv);
    load4<false>((const float*)r.v, i, n, whole, vv);
  }
  if (r.m_out) store4(r.m_out, i, n, whole, mv);
  if (r.v_out) store4(r.v_out, i, n, whole, vv);
}

bool aligned_to(size_t a, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p % a != 0) return false;
  return true;
}

// Deals n tensors out to launches: fill(args, slot, tensor) fills a record, go(args, blocks) launches.
// A tensor has at most 2^33 elements, kMaxBlocks blocks.
template <typename Args, typename Fill, typename Go>
hipError_t for_launches(Args& args, const moe_adamw_tensor* ts, int n, Fill fill, Go go) {
  int slot = 0;
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) {
    if (ts[i].n == 0) continue;
    if (slot == kTensors || (slot && blocks + (ts[i].n + kChunk - 1) / kChunk > kMaxBlocks)) {
      args.count = slot;
      if (hipError_t err = go(args, blocks); err != hipSuccess) return err;
      slot = 0;
      blocks = 0;
    }
    args.start[slot] = (int32_t)blocks;
    fill(args.rec[slot], i);
    blocks += (ts[i].n + kChunk - 1) / kChunk;
    ++slot;
  }
  args.count = slot;
  return slot ? go(args, blocks) : hipSuccess;
}

}  // namespace

hipError_t launch_adamw(const moe_adamw_config& c, const moe_adamw_tensor* ts, int n,
                        hipStream_t st) {
  AdamArgs args;
  args.lr = c.lr;
  args.beta1 = c.beta1;
  args.beta2 = c.beta2;
  args.eps = c.eps;
  args.grad_scale = c.grad_scale;
  args.log_beta1 = log((double)c.beta1);
  args.log_beta2 = log((double)c.beta2);
  args.dynamic = c.dynamic;
  const double t = (double)(c.step < 1 ? 1 : c.step);
  args.rate = (float)((double)c.lr / -expm1(t * args.log_beta1));
  args.inv_root = (float)(1.0 / sqrt(-expm1(t * args.log_beta2)));
  const bool p16 = c.param_dtype == MOE_BF16, g16 = c.grad_dtype == MOE_BF16, q8 = c.state_bits == 8;
  auto fill = [&](AdamRec& r, int i) {
    const moe_adamw_tensor& x = ts[i];
    r = AdamRec{x.param, x.grad, x.m, x.v, x.m_steps, x.v_steps, (bf16_t*)x.copy, x.n, x.weight_decay, 0};
    r.vec = aligned_to(p16 ? 8 : 16, {x.param}) && aligned_to(g16 ? 8 : 16, {x.grad}) &&
            aligned_to(q8 ? 4 : 16, {x.m, x.v}) && aligned_to(8, {x.copy});
  };
  auto launch = [&](auto kern) {
    return for_launches(args, ts, n, fill, [&](const AdamArgs& a, int64_t blocks) {
      hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), 0, st, a);
      return hipGetLastError();
    });
  };
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) bytes += ts[i].n * (16 + (p16 ? 4 : 8) + (g16 ? 2 : 4) + (ts[i].copy ? 2 : 0));
  auto types = [&](auto p, auto g) {
    using P = decltype(p);
    using G = decltype(g);
    return q8                    ? launch(k_adamw<P, G, true, false>)
           : bytes > kStreamBytes ? launch(k_adamw<P, G, false, true>)
                                  : launch(k_adamw<P, G, false, false>);
  };
  if (p16) return g16 ? types(bf16_t{}, bf16_t{}) : types(bf16_t{}, float{});
  return g16 ? types(float{}, bf16_t{}) : types(float{}, float{});
}

hipError_t launch_adamw_moments(const moe_adamw_config& c, const moe_adamw_tensor* ts, int n,
                                float* const* m_out, float* const* v_out, hipStream_t st) {
  MomentArgs args;
  const bool q8 = c.state_bits == 8;
  auto fill = [&](MomentRec& r, int i) {
    const moe_adamw_tensor& x = ts[i];
    r = MomentRec{x.m, x.v, x.m_steps, x.v_steps, m_out ? m_out[i] : nullptr,
                  v_out ? v_out[i] : nullptr, x.n, 0};
    r.vec = aligned_to(q8 ? 4 : 16, {x.m, x.v}) && aligned_to(16, {r.m_out, r.v_out});
  };
  auto launch = [&](auto kern) {
    return for_launches(args, ts, n, fill, [&](const MomentArgs& a, int64_t blocks) {
      hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), 0, st, a);
      return hipGetLastError();
    });
  };
  return q8 ? launch(k_adamw_moments<true>) : launch(k_adamw_moments<false>);
}

}  // namespace moe
