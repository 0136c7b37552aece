// Routing by scores: softmax or sigmoid scores, a selection bias, groups of experts, top-k of the
// biased scores, gates from the unbiased ones.
//
// With l = W_r x + b_r and s_e = softmax(l)_e or 1 / (1 + e^(-l_e)):
//   a_e    = fl32(s_e) + score_bias_e                   what the choice goes by
//   group  = max a or the sum of its two largest a      the best topk_groups groups stay
//   choice = the k largest a of the groups that stay    ties to the lower expert, or group
//   gate   = scale s_e, or scale s_e / (sum of the chosen s)
// The logits are fp64 sums of exact products and the scores are evaluated in fp64, as in the other
// router and for its reason: the choice, and later the fill order of the buffers, turn on the last
// fp32 bits.  a is one fp32 addition, so that a bias that moves in small steps moves it alike on
// every machine.  A gate is rounded once.
//
// Two launches.  k_scored_logits leaves partial logits (fp64, [split][token][expert]) of 16 or 32
// tokens and 16 to 64 experts a block on v_mfma_f64_16x16x4f64; k_scored_choose adds the splits and
// does the rest with 16 lanes a token.  Tokens go through both in chunks, which bounds the workspace.
#include "route_chunks.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- partial logits
// A block of WD x WE waves takes 16 R tokens and 16 EBG WE experts: wave (wd, we) takes expert tiles
// we EBG .. of them and every (S WD)-th quad of 32 columns from quad split WD + wd on.  The waves of
// one we are added in the order of wd, so equal calls give equal bits.  Lane layout of the operands
// and results as in k_route_mfma.
template <typename TIn, int R, int EBG, int WD, int WE>
__global__ __launch_bounds__(64 * WD * WE) void k_scored_logits(
    const TIn* __restrict__ x, const TIn* __restrict__ w, int64_t T, int d, int E, int S,
    int64_t tok_base, int64_t n_tok, double* __restrict__ part) {
  constexpr int kPart = R * EBG * 256;
  __shared__ double lds[WD > 1 ? (WD - 1) * WE * kPart : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int we = wave % WE, wd = wave / WE;
  const int i = lane & 15, q = lane >> 4;
  const int64_t tok0 = (int64_t)blockIdx.x * (16 * R);  // within the chunk
  const int e0 = ((int)blockIdx.y * WE + we) * EBG * 16;
  const int split = blockIdx.z;
  const int d8 = (d + 7) / 8, nq = (d8 + 3) / 4, stride = S * WD;
  const __amdgpu_buffer_rsrc_t xs = buffer_rsrc(x, (uint32_t)(T * d * (int64_t)sizeof(TIn)));
  const __amdgpu_buffer_rsrc_t ws = buffer_rsrc(w, (uint32_t)((int64_t)E * d * sizeof(TIn)));

  f64x4_t acc[R][EBG];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int b = 0; b < EBG; ++b) acc[r][b] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  Chunk8<TIn> xr[R], wr[EBG];
  auto load = [&](int cq) {
    const int c = cq * 4 + q;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = tok0 + 16 * r + i;
      xr[r].load(xs, cq < nq && t < n_tok, tok_base + t, c, d);
    }
#pragma unroll
    for (int b = 0; b < EBG; ++b) {
      const int e = e0 + 16 * b + i;
      wr[b].load(ws, cq < nq && e < E, e, c, d);
    }
  };
  int cq = split * WD + wd;
  load(cq);
  for (; cq < nq; cq += stride) {
    double xa[R][8], wb[EBG][8];
#pragma unroll
    for (int r = 0; r < R; ++r) xr[r].widen(xa[r]);
#pragma unroll
    for (int b = 0; b < EBG; ++b) wr[b].widen(wb[b]);
    load(cq + stride);
#pragma unroll
    for (int s8 = 0; s8 < 8; ++s8)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int b = 0; b < EBG; ++b)
          acc[r][b] = __builtin_amdgcn_mfma_f64_16x16x4f64(xa[r][s8], wb[b][s8], acc[r][b], 0, 0, 0);
  }
  if constexpr (WD > 1) {
    if (wd > 0) {
      double* mine = lds + ((wd - 1) * WE + we) * kPart;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int b = 0; b < EBG; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) mine[((r * EBG + b) * 4 + j) * 64 + lane] = acc[r][b][j];
    }
    __syncthreads();
    if (wd > 0) return;
    for (int o = 1; o < WD; ++o) {
      const double* other = lds + ((o - 1) * WE + we) * kPart;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int b = 0; b < EBG; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r][b][j] += other[((r * EBG + b) * 4 + j) * 64 + lane];
    }
  }
  // lane l, register j of a tile holds token 4 j + l / 16, expert l % 16 of the tile
  double* out = part + (int64_t)split * n_tok * E;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int b = 0; b < EBG; ++b) {
      const int e = e0 + 16 * b + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = tok0 + 16 * r + 4 * j + q;
        if (e < E && t < n_tok) out[t * E + e] = acc[r][b][j];
      }
    }
}

// ---------------------------------------------------------------- scores and choice
struct ChooseArgs {
  const double* part;  // [S][n_tok][E]
  int S;
  int64_t tok_base, n_tok;
  int E, k;
  int sigmoid, n_groups, topk_groups, top2, renormalize;
  double scale;
  const float* b_router;    // may be NULL, as all below but ids and gates
  const float* score_bias;
  const uint8_t* mask;
  int32_t* ids;
  float* gates;
  float* logits;
};

// The order of floats as the order of unsigned numbers: NaN above everything, 0 is no float's.
__device__ __forceinline__ uint32_t order_key(float a) {
  const uint32_t u = __float_as_uint(a);
  return a != a ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// A key below this is no candidate's (order_key(-FLT_MAX)): 0 for one that is off or out, 1 + c for the
// one that choice c took.
constexpr uint32_t kLeastKey = 0x00800000u;

// Reductions over a row of 16 lanes, in the order xor 8, 4, 2, 1; every lane gets the result.
template <typename Op>
__device__ __forceinline__ double row16(double v, Op op) {
#pragma unroll
  for (int s = 8; s >= 1; s >>= 1)
    v = op(v, __longlong_as_double((long long)xor_partner((uint64_t)__double_as_longlong(v), s)));
  return v;
}
__device__ __forceinline__ uint64_t row16_max(uint64_t v) {
#pragma unroll
  for (int s = 8; s >= 1; s >>= 1) {
    const uint64_t o = xor_partner(v, s);
    v = o > v ? o : v;
  }
  return v;
}

// 16 lanes a token, lane l of them holds experts l, l + 16, ... (NV of them).  The lanes of a token
// share its row of keys in LDS only where there are groups.
template <int NV>
__global__ __launch_bounds__(256) void k_scored_choose(const ChooseArgs a) {
  extern __shared__ uint32_t shared_keys[];  // groups: [16 tokens][E + n_groups]
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t t = (int64_t)blockIdx.x * 16 + row;
  const bool there = t < a.n_tok;
  const int64_t tt = a.tok_base + t;
  const bool real = there && (!a.mask || a.mask[tt]);
  const int E = a.E, k = a.k;
  auto add = [](double u, double v) { return u + v; };
  auto larger = [](double u, double v) { return fmax(u, v); };

  double z[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) z[i] = 0.0;
  if (real) {
    const double* p = a.part + t * E;
    for (int s = 0; s < a.S; ++s, p += a.n_tok * E)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * 16 + l < E) z[i] += p[i * 16 + l];
    if (a.b_router)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * 16 + l < E) z[i] += (double)a.b_router[i * 16 + l];
  }
  if (there && a.logits)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * 16 + l < E) a.logits[tt * E + i * 16 + l] = (float)z[i];

  // scores in place of the logits: p[i], 0 past E
  double p[NV];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = i * 16 + l < E ? 1.0 / (1.0 + exp(-z[i])) : 0.0;
  } else {
    double m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * 16 + l < E) m = fmax(m, z[i]);
    m = row16(m, larger);
    if (m == -INFINITY) m = 0.0;  // nothing but -inf (and NaN, which fmax leaves out): zeros
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = i * 16 + l < E ? exp(z[i] - m) : 0.0;
      sum += p[i];
    }
    sum = row16(sum, add);
    if (sum == 0.0) sum = 1.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = p[i] / sum;
  }

  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * 16 + l;
    key[i] = 0;
    if (e < E) {
      float v = (float)p[i];
      bool off = false;
      if (a.score_bias) {
        const float b = a.score_bias[e];
        off = b == -INFINITY;
        v += b;
      }
      if (!off) key[i] = order_key(v);
    }
  }

  if (a.topk_groups < a.n_groups) {  // uniform over the grid
    const int G = a.n_groups, gs = E / G;
    uint32_t* keys = shared_keys + row * (E + G);
    uint32_t* group = keys + E;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * 16 + l < E) keys[i * 16 + l] = key[i];
    __syncthreads();
    for (int g = l; g < G; g += 16) {
      uint32_t best = 0, second = 0;
      for (int j = 0; j < gs; ++j) {
        const uint32_t v = keys[g * gs + j];
        const uint32_t low = v < best ? v : best;
        best = v > best ? v : best;
        second = low > second ? low : second;
      }
      // one expert that is on speaks for its group alone; a group without any is the last
      group[g] = a.top2 && second ? order_key(key_value(best) + key_value(second)) : best;
    }
    __syncthreads();
    // a group stays if fewer than topk_groups are better (or as good and before it)
    for (int g = l; g < G; g += 16) {
      const uint32_t mine = group[g];
      int better = 0;
      for (int o = 0; o < G; ++o) better += group[o] > mine || (group[o] == mine && o < g);
      keys[g] = better < a.topk_groups;  // the experts' keys are in registers
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * 16 + l < E && !keys[(i * 16 + l) / gs]) key[i] = 0;
  }

  int taken = 0;
  if (real)
    for (; taken < k; ++taken) {
      uint32_t best = 0, at = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (key[i] > best) {
          best = key[i];
          at = i;
        }
      const uint64_t win =
          row16_max(((uint64_t)best << 32) | (0xFFFFFFFFu - (at * 16 + (uint32_t)l)));
      if ((uint32_t)(win >> 32) < kLeastKey) break;  // all 16 lanes agree
      const uint32_t e = 0xFFFFFFFFu - (uint32_t)win;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (e == (uint32_t)(i * 16 + l)) key[i] = 1 + taken;
    }
  if (!there) return;

  auto chosen = [&](int i) { return key[i] != 0 && key[i] < kLeastKey; };
  double total = 1.0;
  if (a.renormalize) {
    total = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (chosen(i)) total += p[i];
    total = row16(total, add);
    // Scores that the range of fp64 has lost, or nearly: e^l instead, from the largest chosen logit
    // (1 + e^l is 1 there); all of them zero (-inf): the gates are zero.
    if (total < 1e-280) {
      double m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (chosen(i)) m = fmax(m, z[i]);
      m = row16(m, larger);
      if (m == -INFINITY) m = 0.0;
      total = 0.0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (chosen(i)) {
          p[i] = exp(z[i] - m);
          total += p[i];
        }
      total = row16(total, add);
      if (total == 0.0) total = 1.0;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (chosen(i)) {
      const int64_t at = tt * k + (key[i] - 1);
      a.ids[at] = i * 16 + l;
      a.gates[at] = (float)(a.scale * (p[i] / total));
    }
  for (int c = taken + l; c < k; c += 16) {  // masked, or too few experts are on
    a.ids[tt * k + c] = -1;
    a.gates[tt * k + c] = 0.0f;
  }
}

// ---------------------------------------------------------------- launches
struct Plan {
  int64_t chunk;  // tokens that go through the two launches at a time
  int S;          // splits of the columns
  bool large;
};

// At most 64 MiB of partial logits.  Short batches take 16 x 16 tiles and split the columns until
// there are some hundred blocks; long ones 32 x 32 tiles, which widen each value for two products.
Plan plan(const moe_shape& s) {
  Plan p;
  p.large = s.T >= 4096;
  const int nq = ((s.d_model + 7) / 8 + 3) / 4;
  if (p.large) {
    p.S = 1;
    p.chunk = ((int64_t)64 << 20) / (8 * s.n_experts) / 32 * 32;
  } else {
    const int64_t tiles = (s.T + 15) / 16 * ((s.n_experts + 15) / 16);
    const int most = (nq + 7) / 8;
    p.S = (int)(512 / (tiles > 0 ? tiles : 1));
    p.S = p.S < 1 ? 1 : p.S > 8 ? 8 : p.S;
    p.S = p.S < most ? p.S : most;
    p.chunk = 4096;
  }
  if (p.chunk > s.T) p.chunk = s.T;
  return p;
}

template <typename TIn, int R, int EBG, int WD, int WE>
hipError_t launch_logits(const moe_shape& s, const TIn* x, const TIn* w, const Plan& p,
                         int64_t base, int64_t n, double* part, hipStream_t st) {
  const dim3 grid((unsigned)((n + 16 * R - 1) / (16 * R)),
                  (unsigned)((s.n_experts + 16 * EBG * WE - 1) / (16 * EBG * WE)), (unsigned)p.S);
  hipLaunchKernelGGL((k_scored_logits<TIn, R, EBG, WD, WE>), grid, dim3(64 * WD * WE), 0, st, x, w,
                     s.T, s.d_model, s.n_experts, p.S, base, n, part);
  return hipGetLastError();
}

template <typename TIn>
hipError_t logits_any(const moe_shape& s, const TIn* x, const TIn* w, const Plan& p, int64_t base,
                      int64_t n, double* part, hipStream_t st) {
  if (!p.large) return launch_logits<TIn, 1, 1, 8, 1>(s, x, w, p, base, n, part, st);
  if (s.n_experts <= 16) return launch_logits<TIn, 2, 1, 4, 1>(s, x, w, p, base, n, part, st);
  if (s.n_experts <= 32) return launch_logits<TIn, 2, 2, 4, 1>(s, x, w, p, base, n, part, st);
  return launch_logits<TIn, 2, 2, 4, 2>(s, x, w, p, base, n, part, st);
}

hipError_t launch_choose(const ChooseArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.n_tok + 15) / 16));
  const size_t lds = a.topk_groups < a.n_groups ? (size_t)16 * 4 * (a.E + a.n_groups) : 0;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), lds, st, a);
    return hipGetLastError();
  };
  if (a.E <= 16) return go(k_scored_choose<1>);
  if (a.E <= 32) return go(k_scored_choose<2>);
  if (a.E <= 64) return go(k_scored_choose<4>);
  if (a.E <= 128) return go(k_scored_choose<8>);
  return go(k_scored_choose<16>);
}

}  // namespace

size_t route_scored_ws_bytes(const moe_shape& s) {
  const Plan p = plan(s);
  return ((size_t)p.S * p.chunk * s.n_experts * 8 + 255) & ~(size_t)255;
}

hipError_t launch_route_scored(const moe_shape& s, const moe_routing& r, const void* x,
                               const void* w_router, const float* b_router,
                               const float* score_bias, const uint8_t* mask, int32_t* ids,
                               float* gates, float* logits, void* ws, hipStream_t st) {
  const Plan p = plan(s);
  double* part = (double*)ws;
  for (int64_t base = 0; base < s.T; base += p.chunk) {
    const int64_t n = s.T - base < p.chunk ? s.T - base : p.chunk;
    hipError_t err = s.dtype == MOE_BF16
                         ? logits_any<bf16_t>(s, (const bf16_t*)x, (const bf16_t*)w_router, p, base,
                                              n, part, st)
                         : logits_any<float>(s, (const float*)x, (const float*)w_router, p, base, n,
                                             part, st);
    if (err != hipSuccess) return err;
    ChooseArgs a{part, p.S, base, n, s.n_experts, s.top_k, r.score == MOE_SCORE_SIGMOID,
                 r.n_groups, r.topk_groups, r.group_score == MOE_GROUP_TOP_TWO, r.renormalize,
                 (double)r.scale, b_router, score_bias, mask, ids, gates, logits};
    if ((err = launch_choose(a, st)) != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
