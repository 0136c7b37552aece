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
// zero keeps a code of 1 at least.  Rounding to nearest, so that equal calls give equal bits and the
// codes are the same wherever they are computed: of Gaussian gradients whose size varies by e^(+-1)
// within a block, r stays within 1.1 % of fp32's on average at beta2 0.95 and 5.2 % at 0.999 (steps 201
// to 4000).  Its price: a step that takes less than half a code off does nothing.  Beside a largest
// value that stays, m's codes with c (1 - sqrt(beta1)) <= 1/2 (9 at 0.9, 0.5 % of the largest) and r's
// with c (1 - beta2^(1/4)) <= 1/2 (39 at 0.95; all at 0.999) do not decay, and an element whose gradient
// ends in a block where others go on keeps moving: with a gradient of 0.004 for 200 steps beside N(0, 1)
// and none for 2000 more (lr 1e-3), by 0.47 at beta2 0.95 and 0.15 at 0.999, against 0.012 and 0.009 with
// fp32 moments.  A block whose gradients end together decays as it should, by its steps.
//
// Bound: memory, 28 bytes an element for fp32 moments and gradients, 14 to 18 for 8 bits: 268 million
// elements with bf16 gradients 1145 to 1220 us (5.7 to 6.1 TB/s), 37.8 million at 8 bits with copies 105
// us (5.7 TB/s; with each load behind the branch for odd tensors 115).  The tensors' addresses go along
// as kernel arguments, 64 or 48 to a launch; a block takes 1024 elements of one tensor, a thread 4
// neighbours, so that a wave has exactly the 256 that share a step.
#include <math.h>

#include <type_traits>

#include "math_f64.h"

namespace moe {

namespace {

constexpr int kTensors32 = 64, kTensors8 = 48;  // a launch, whose arguments stay below 4 KiB
constexpr int kChunk = 1024;    // elements a block (loops over 2048 and 4096 took 3 and 5 % longer)
constexpr int64_t kMaxBlocks = 1 << 23;  // a launch: 2^32 threads are too many
// From this many bytes on a pass, more than the last-level cache holds, 32-bit moments and what goes with
// them are loaded past the caches (1148 us against 1248 for 268 million elements, but 22.8 against 19.8 for
// 4.2 million, where all of it stays in the cache from step to step).
constexpr int64_t kStreamBytes = (int64_t)256 << 20;
constexpr int kQuantBlock = 256;
static_assert(kChunk == 4 * 256, "a block's threads take 4 elements each");

struct AdamRec32 {
  void* p;
  const void* g;
  void* m;
  void* v;
  bf16_t* copy;
  int64_t n;
  float wd;
  int vec;  // every array lies where 4 elements load at once
};
struct AdamRec8 : AdamRec32 {
  float* m_steps;
  float* v_steps;
};
template <typename Rec_, int N>
struct AdamArgs {
  typedef Rec_ Rec;
  static constexpr int kTensors = N;
  Rec rec[N];
  int32_t start[N];  // first chunk of each tensor
  int32_t count;
  float lr, beta1, beta2, eps, grad_scale, rate, inv_root;
  double log_beta1, log_beta2;
  const float* dynamic;
};
typedef AdamArgs<AdamRec32, kTensors32> AdamArgs32;
typedef AdamArgs<AdamRec8, kTensors8> AdamArgs8;
static_assert(sizeof(AdamArgs32) <= 4096 && sizeof(AdamArgs8) <= 4096, "kernel arguments");

struct Rates {
  float lr, grad_scale, rate, inv_root;
};

// The 4 elements of a lane, as loaded.
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <bool WHOLE, bool STREAM>
__device__ __forceinline__ void load4(const float* p, int64_t i, int64_t n, float (&o)[4]) {
  if constexpr (WHOLE) {
    const f32x4* at = reinterpret_cast<const f32x4*>(p + i);
    const f32x4 f = STREAM ? __builtin_nontemporal_load(at) : *at;
    o[0] = f[0], o[1] = f[1], o[2] = f[2], o[3] = f[3];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = i + j < n ? p[i + j] : 0.0f;
  }
}
template <bool WHOLE, bool STREAM>
__device__ __forceinline__ void load4(const bf16_t* p, int64_t i, int64_t n, float (&o)[4]) {
  if constexpr (WHOLE) {
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
template <bool WHOLE>
__device__ __forceinline__ void store4(float* p, int64_t i, int64_t n, const float (&o)[4]) {
  if constexpr (WHOLE) {
    const f32x4 w = {o[0], o[1], o[2], o[3]};
    __builtin_nontemporal_store(w, reinterpret_cast<f32x4*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = o[j];
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store4(bf16_t* p, int64_t i, int64_t n, const float (&o)[4]) {
  const uint32_t a = pack_bf16x2(o[0], o[1]), b = pack_bf16x2(o[2], o[3]);
  if constexpr (WHOLE) {
    __builtin_nontemporal_store((uint64_t)b << 32 | a, reinterpret_cast<uint64_t*>(p + i));
  } else {
    const bf16_t w[4] = {(bf16_t)a, (bf16_t)(a >> 16), (bf16_t)b, (bf16_t)(b >> 16)};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = w[j];
  }
}
// 4 codes in a dword, the first lowest
template <bool WHOLE>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int64_t n) {
  if constexpr (WHOLE) return *reinterpret_cast<const uint32_t*>(p + i);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) w |= (uint32_t)p[i + j] << (8 * j);
  return w;
}
template <bool WHOLE>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, uint32_t w) {
  if constexpr (WHOLE) {
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

// Four elements of a lane.  WHOLE: the chunk is inside the tensor and its arrays lie where 4 elements
// load at once; decided once a chunk, so that no load waits behind a branch for the one before.
template <bool WHOLE, typename P, typename G, bool Q8, bool STREAM, typename Args>
__device__ __forceinline__ void adamw_lane(const Args& a, const typename Args::Rec& r, const Rates& c,
                                           int64_t i, int64_t n) {
  P* p = (P*)r.p;
  const G* g = (const G*)r.g;
  bf16_t* copy = r.copy;
  const float lr_wd = c.lr * r.wd;
  float pv[4], gv[4], mv[4], vv[4];
  const int64_t qb = i / kQuantBlock;
  if constexpr (Q8) {
    const uint32_t mw = load_codes<WHOLE>((const uint8_t*)r.m, i, n);
    const uint32_t vw = load_codes<WHOLE>((const uint8_t*)r.v, i, n);
    const float ms = r.m_steps[qb], vs = r.v_steps[qb];
    load4<WHOLE, STREAM>(p, i, n, pv);
    load4<WHOLE, STREAM>(g, i, n, gv);
    decode_m(mw, ms, mv);
    decode_v(vw, vs, vv);
  } else {
    load4<WHOLE, STREAM>(p, i, n, pv);
    load4<WHOLE, STREAM>(g, i, n, gv);
    load4<WHOLE, STREAM>((const float*)r.m, i, n, mv);
    load4<WHOLE, STREAM>((const float*)r.v, i, n, vv);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) moments(gv[j] * c.grad_scale, a.beta1, a.beta2, mv[j], vv[j]);
  float rv[4];
  if constexpr (Q8) {
    // The kernel of 8 bits is short of instructions before it is of bytes (122 an element with every root
    // and quotient in full: 139 us against 128 for 37.8 million elements, before its stores and loads
    // were what they are): roots and the quotient to a step of fp32, except roots of denormal
    // numbers, which the instruction takes for zeros.
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
  store4<WHOLE>(p, i, n, pv);
  if (copy) store4<WHOLE>(copy, i, n, pv);
  if constexpr (Q8) {
    // elements past the tensor's end are zeros; the largest root is the largest v's
    const float ms = wave_absmax<true>(mv) / 16129.0f, vs = sqrtf(wave_absmax<false>(vv)) / 65025.0f;
    const uint32_t mc = encode4<127>(mv, [&](int j) { return mv[j]; }, ms);
    const uint32_t vc = encode4<255>(rv, [&](int j) { return sqrtf(vv[j]); }, vs);
    store_codes<WHOLE>((uint8_t*)r.m, i, n, mc);
    store_codes<WHOLE>((uint8_t*)r.v, i, n, vc);
    if ((threadIdx.x & 63) == 0) {
      r.m_steps[qb] = ms;
      r.v_steps[qb] = vs;
    }
  } else {
    store4<WHOLE>((float*)r.m, i, n, mv);
    store4<WHOLE>((float*)r.v, i, n, vv);
  }
}

// One chunk of kChunk elements.
template <typename P, typename G, bool Q8, bool STREAM, typename Args>
__device__ __forceinline__ void adamw_chunk(const Args& a, const Rates& c, int chunk) {
  const int ti = tensor_of(a.start, a.count, chunk);
  const typename Args::Rec& r = a.rec[ti];
  const int64_t n = r.n, base = (int64_t)(chunk - a.start[ti]) * kChunk;
  const int64_t i = base + (int64_t)threadIdx.x * 4;
  if (r.vec && base + kChunk <= n)
    adamw_lane<true, P, G, Q8, STREAM>(a, r, c, i, n);
  else if (base + (threadIdx.x & ~63) * 4 < n)  // waves that hold nothing leave together
    adamw_lane<false, P, G, Q8, STREAM>(a, r, c, i, n);
}

// A chunk a block.
template <typename P, typename G, bool Q8, bool STREAM, typename Args>
__global__ __launch_bounds__(256) void k_adamw(const Args a) {
  adamw_chunk<P, G, Q8, STREAM>(a, Rates{a.lr, a.grad_scale, a.rate, a.inv_root}, (int)blockIdx.x);
}

// The same with rates from the device.  A correction 1 - beta^t is 1 - e^y in fp64, y = t log beta: as
// near as 2^-53 / |y|, and |y| is 2^-24 at least.  All waves form both (some 70 instructions; the general
// functions, 200, in as many blocks as run at once with several chunks each: 137 us against 113 for 37.8
// million elements at 8 bits, 1459 against 1244 for 268 million at 32).
template <typename P, typename G, bool Q8, bool STREAM, typename Args>
__global__ __launch_bounds__(256) void k_adamw_dynamic(const Args a) {
  if (a.dynamic[3] != 0.0f) return;
  const double t = fmax((double)a.dynamic[2], 1.0);
  const double c1 = 1.0 - exp_clamped(t * a.log_beta1), c2 = 1.0 - exp_clamped(t * a.log_beta2);
  double root = __builtin_amdgcn_rsq(c2);
  root = root * fma(-0.5 * c2 * root, root, 1.5);
  Rates c;
  c.lr = a.dynamic[0];
  c.grad_scale = a.dynamic[1];
  c.rate = (float)((double)c.lr / c1);
  c.inv_root = (float)root;
  adamw_chunk<P, G, Q8, STREAM>(a, c, (int)blockIdx.x);
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
  typedef MomentRec Rec;
  static constexpr int kTensors = kTensors8;
  MomentRec rec[kTensors];
  int32_t start[kTensors];
  int32_t count;
};
static_assert(sizeof(MomentArgs) <= 4096, "kernel arguments");

template <bool WHOLE, bool Q8>
__device__ __forceinline__ void moments_lane(const MomentRec& r, int64_t i, int64_t n) {
  float mv[4], vv[4];
  if constexpr (Q8) {
    const uint32_t mw = load_codes<WHOLE>((const uint8_t*)r.m, i, n);
    const uint32_t vw = load_codes<WHOLE>((const uint8_t*)r.v, i, n);
    const float ms = r.m_steps[i / kQuantBlock], vs = r.v_steps[i / kQuantBlock];
    decode_m(mw, ms, mv);
    decode_v(vw, vs, vv);
  } else {
    load4<WHOLE, false>((const float*)r.m, i, n, mv);
    load4<WHOLE, false>((const float*)r.v, i, n, vv);
  }
  if (r.m_out) store4<WHOLE>(r.m_out, i, n, mv);
  if (r.v_out) store4<WHOLE>(r.v_out, i, n, vv);
}

template <bool Q8>
__global__ __launch_bounds__(256) void k_adamw_moments(const MomentArgs a) {
  const int ti = tensor_of(a.start, a.count, (int)blockIdx.x);
  const MomentRec& r = a.rec[ti];
  const int64_t n = r.n, base = (int64_t)((int)blockIdx.x - a.start[ti]) * kChunk;
  const int64_t i = base + (int64_t)threadIdx.x * 4;
  if (r.vec && base + kChunk <= n)
    moments_lane<true, Q8>(r, i, n);
  else if (i < n)
    moments_lane<false, Q8>(r, i, n);
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
    if (slot == Args::kTensors || (slot && blocks + (ts[i].n + kChunk - 1) / kChunk > kMaxBlocks)) {
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
  const bool p16 = c.param_dtype == MOE_BF16, g16 = c.grad_dtype == MOE_BF16, q8 = c.state_bits == 8;
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) bytes += ts[i].n * (16 + (p16 ? 4 : 8) + (g16 ? 2 : 4) + (ts[i].copy ? 2 : 0));
  auto launch = [&](auto args, auto kern, auto dynamic_kern) {
    typedef typename decltype(args)::Rec Rec;
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
    auto fill = [&](Rec& r, int i) {
      const moe_adamw_tensor& x = ts[i];
      r.p = x.param, r.g = x.grad, r.m = x.m, r.v = x.v, r.copy = (bf16_t*)x.copy;
      r.n = x.n, r.wd = x.weight_decay;
      r.vec = aligned_to(p16 ? 8 : 16, {x.param}) && aligned_to(g16 ? 8 : 16, {x.grad}) &&
              aligned_to(q8 ? 4 : 16, {x.m, x.v}) && aligned_to(8, {x.copy});
      if constexpr (std::is_same<Rec, AdamRec8>::value) r.m_steps = x.m_steps, r.v_steps = x.v_steps;
    };
    return for_launches(args, ts, n, fill, [&](const auto& a, int64_t blocks) {
      hipLaunchKernelGGL(c.dynamic ? dynamic_kern : kern, dim3((unsigned)blocks), dim3(256), 0, st, a);
      return hipGetLastError();
    });
  };
  auto types = [&](auto p, auto g) {
    using P = decltype(p);
    using G = decltype(g);
    if (q8)
      return launch(AdamArgs8{}, k_adamw<P, G, true, false, AdamArgs8>,
                    k_adamw_dynamic<P, G, true, false, AdamArgs8>);
    return bytes > kStreamBytes ? launch(AdamArgs32{}, k_adamw<P, G, false, true, AdamArgs32>,
                                         k_adamw_dynamic<P, G, false, true, AdamArgs32>)
                                : launch(AdamArgs32{}, k_adamw<P, G, false, false, AdamArgs32>,
                                         k_adamw_dynamic<P, G, false, false, AdamArgs32>);
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
