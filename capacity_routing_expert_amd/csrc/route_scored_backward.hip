// Backward pass of routing by scores: from the gradient on the gates to the gradient on the logits.
//
// With S the choices c of a token, s_c their scores, q_c = s_c / sum_S s (renormalised gates / scale):
//   renormalised:  h_c = scale (dg_c - sum_S dg q) q_c,   softmax: dl += h_c at c's expert,
//                                                         sigmoid: dl += h_c (1 - s_c)
//   otherwise:     sigmoid: dl += scale dg_c s_c (1 - s_c) at c's expert
//                  softmax: dl_e = s_e (u_e - sum_S u s), u_e the sum of scale dg_c over e's choices
// (renormalised softmax gates depend on the chosen logits alone: the rest of the row cancels.)
// So only a softmax that is not renormalised reads whole rows of logits; the rest reads the chosen
// ones.  q_c is formed from e^(l_c - M), M the largest chosen logit or 0 if that is less: it stays
// exact where the scores themselves leave the range of fp32.
//
// Bound: writing dlogits, 4 bytes an expert and token, and reading as much where the row or
// dlogits_add comes in.  One launch; the 16 lanes of a RouterRow hold a token.
#include "router_rows.h"

namespace moe {

namespace {

struct ScoredBackArgs {
  const float* logits;
  const int32_t* ids;
  const float* dgates;
  const float* add;     // may be NULL, or dlogits
  const uint8_t* mask;  // may be NULL
  float* dlogits;
  int64_t T;
  int E, k;
  float scale;
};

// Between LDS accesses of a wave's lanes to each other's places: the hardware keeps a wave's order, this
// keeps the compiler to it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// e^x for x <= 0 (or NaN) down to the least denormal number: exp_nonpositive with results below 2^-126,
// which the exponential instruction leaves out, formed 64 binary places higher.
__device__ __forceinline__ float exp_to_denormal(float x) {
  const float kHi = 1.44269502162933349609375f, kLo = 1.92596299e-8f, kLn2 = 0.693147182f;
  const float t = x * kHi;
  const float r = fmaf(x, kHi, -t) + x * kLo;
  const bool low = t < -125.0f;
  const float v = __builtin_amdgcn_exp2f(low ? t + 64.0f : t);
  const float e = fmaf(v, r * kLn2, v) * (low ? 0x1p-64f : 1.0f);
  return x < -104.0f ? 0.0f : e;
}

// e^-|l| and from it sigmoid(l), sigmoid(-l)
struct Sigmoid {
  float s, rest;
  __device__ __forceinline__ explicit Sigmoid(float l) {
    const float a = exp_to_denormal(-fabsf(l)), big = 1.0f / (1.0f + a), small = a * big;
    s = l >= 0.0f ? big : small;
    rest = l >= 0.0f ? small : big;
    if (l != l) s = rest = l;
  }
};

// One choice of a token: its expert (-1: none), logit and gate gradient.
struct Choice {
  int id;
  float l, dg;
};
__device__ __forceinline__ Choice load_choice(const ScoredBackArgs& a, int64_t t, int c) {
  Choice v{-1, 0.0f, 0.0f};
  if (c < a.k) {
    v.id = a.ids[t * a.k + c];
    if ((unsigned)v.id >= (unsigned)a.E) v.id = -1;
    if (v.id >= 0) {
      v.dg = a.dgates[t * a.k + c];
      v.l = a.logits[t * a.E + v.id];
    }
  }
  return v;
}

// Row::softmax with probabilities down to the least denormal number.
template <typename Row>
__device__ __forceinline__ void row_softmax(float (&v)[Row::NV]) {
  float m = v[0], s = 0.0f;
#pragma unroll
  for (int i = 1; i < Row::NV; ++i) m = fmaxf(m, v[i]);
  m = row_max<Row::LPT>(m);
  m = m == -INFINITY ? 0.0f : m;
#pragma unroll
  for (int i = 0; i < Row::NV; ++i) {
    v[i] = exp_to_denormal(v[i] - m);
    s += v[i];
  }
  s = row_sum<Row::LPT>(s);
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < Row::NV; ++i) v[i] *= inv;
}

template <typename Row, bool SIGMOID, bool RENORM>
__global__ __launch_bounds__(256) void k_scored_back(const ScoredBackArgs a) {
  constexpr int LPT = Row::LPT, NV = Row::NV, TPB = 256 / LPT;
  constexpr bool LDS = NV >= 8;
  __shared__ float shared_rows[LDS ? TPB : 1][LDS ? LPT * NV : 1];
  const int l = threadIdx.x % LPT;
  const int64_t t = (int64_t)blockIdx.x * TPB + threadIdx.x / LPT;
  if (t >= a.T) return;  // all lanes of a token together
  float dl[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) dl[i] = 0.0f;
  if (a.mask && !a.mask[t]) {
    Row::store(a.dlogits + t * a.E, a.E, l, dl);
    return;
  }

  // the choices' maximum and sums, LPT choices at a time; the first LPT stay in registers
  const Choice first = load_choice(a, t, l);
  auto choice = [&](int c0) { return c0 == 0 ? first : load_choice(a, t, c0 + l); };
  float m = -INFINITY, den = 0.0f, num = 0.0f;
  if constexpr (RENORM) {
    for (int c0 = 0; c0 < a.k; c0 += LPT) {
      const Choice v = choice(c0);
      if (v.id >= 0) m = fmaxf(m, v.l);
    }
    m = row_max<LPT>(m);
    if (SIGMOID) m = fminf(m, 0.0f);
    if (m == -INFINITY) m = 0.0f;  // every chosen score is zero: so are the shares below
  }
  // the share of a choice before it is divided by their sum
  auto weight = [&](const Choice& v) {
    if (v.id < 0) return 0.0f;
    if (!SIGMOID) return v.l <= m ? exp_to_denormal(v.l - m) : v.l - m + 1.0f;  // NaN (and inf) go on
    const Sigmoid s(v.l);
    return v.l > m ? s.s : exp_to_denormal(v.l - m) * s.rest;
  };
  if constexpr (RENORM) {
    for (int c0 = 0; c0 < a.k; c0 += LPT) {
      const Choice v = choice(c0);
      const float w = weight(v);
      den += w;
      num += w * v.dg;
    }
    den = row_sum<LPT>(den);
    num = row_sum<LPT>(num);
  }
  const float inv = den == 0.0f ? 0.0f : 1.0f / den, mean = num * inv;

  float p[NV];
  if constexpr (!SIGMOID && !RENORM) {
    Row::load(a.logits + t * a.E, a.E, l, -INFINITY, p);
    row_softmax<Row>(p);
  }
  auto part = [&](const Choice& v) {
    float h;
    if constexpr (RENORM) {
      h = a.scale * (weight(v) * inv) * (v.dg - mean);
      if (SIGMOID) h *= Sigmoid(v.l).rest;
    } else {
      h = a.scale * v.dg;
      if (SIGMOID) {
        const Sigmoid s(v.l);
        h *= s.s * s.rest;
      }
    }
    return h;
  };
  // Every choice's part to the lane that holds its expert.  Through the token's row in LDS, where a lane
  // a choice writes and the row's lanes read (T 32771, E 256, top-8 of renormalised sigmoids: 15.9 us
  // with the moves below, 10.3 so); the lanes of a token are in one wave, whose LDS accesses keep
  // their order.  An expert that a token holds twice, or more choices than lanes: lane moves, in
  // choice order.
  bool moves = !LDS || a.k > LPT;
  if constexpr (LDS) {
    float* row = shared_rows[threadIdx.x / LPT];
    if (!moves) {
#pragma unroll
      for (int i = 0; i < NV; ++i) row[l * NV + i] = 0.0f;
      wave_sync();
      const float mine = (float)(l + 1);
      if (first.id >= 0) row[first.id] = mine;
      wave_sync();
      const bool lost = first.id >= 0 && row[first.id] != mine;  // another choice of the same expert
      wave_sync();
      moves = row_max<LPT>(lost ? 1.0f : 0.0f) > 0.0f;
      if (!moves) {
        const float h = part(first);
        if (first.id >= 0) row[first.id] = h;
        wave_sync();
#pragma unroll
        for (int i = 0; i < NV; ++i) dl[i] = Row::expert(l, i) < a.E ? row[Row::expert(l, i)] : 0.0f;
      }
    }
  }
  if (moves)
    for (int c0 = 0; c0 < a.k; c0 += LPT) {
      const Choice v = choice(c0);
      const float h = part(v);
      const int n = a.k - c0 < LPT ? a.k - c0 : LPT;
      for (int j = 0; j < n; ++j) {
        const int id = __shfl(v.id, j, LPT);
        const float hj = __shfl(h, j, LPT);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (id == Row::expert(l, i)) dl[i] += hj;  // experts past E are no choice's
      }
    }
  if constexpr (!SIGMOID && !RENORM) {
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) dot += p[i] * dl[i];
    dot = row_sum<LPT>(dot);
#pragma unroll
    for (int i = 0; i < NV; ++i) dl[i] = p[i] * (dl[i] - dot);
  }
  if (a.add) {
    float add[NV];
    Row::load(a.add + t * a.E, a.E, l, 0.0f, add);
#pragma unroll
    for (int i = 0; i < NV; ++i) dl[i] += add[i];
  }
  Row::store(a.dlogits + t * a.E, a.E, l, dl);
}

}  // namespace

hipError_t launch_route_scored_backward(const moe_shape& s, const moe_routing& r,
                                        const float* logits, const int32_t* ids,
                                        const float* dgates, const float* add, const uint8_t* mask,
                                        float* dlogits, hipStream_t st) {
  const uintptr_t all = (uintptr_t)logits | (uintptr_t)add | (uintptr_t)dlogits;
  const bool vec = s.n_experts % 4 == 0 && all % 16 == 0;
  constexpr int64_t kTokens = 1 << 27;  // a launch: up to 16 threads each, and 2^32 are too many
  for (int64_t t = 0; t < s.T; t += kTokens) {
    const int64_t n = s.T - t < kTokens ? s.T - t : kTokens, e = t * s.n_experts, c = t * s.top_k;
    const ScoredBackArgs a{logits + e, ids + c, dgates + c, add ? add + e : nullptr,
                           mask ? mask + t : nullptr, dlogits + e, n, s.n_experts, s.top_k, r.scale};
    const hipError_t err = with_router_row(s.n_experts, vec, [&](auto row) {
      using Row = decltype(row);
      const dim3 grid((unsigned)((n + 256 / Row::LPT - 1) / (256 / Row::LPT)));
      auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, a);
        return hipGetLastError();
      };
      if (r.score == MOE_SCORE_SIGMOID)
        return r.renormalize ? go(k_scored_back<Row, true, true>) : go(k_scored_back<Row, true, false>);
      return r.renormalize ? go(k_scored_back<Row, false, true>) : go(k_scored_back<Row, false, false>);
    });
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
