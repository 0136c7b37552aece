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
// tokens and 16 or 32 experts a block on v_mfma_f64_16x16x4f64, k_scored_logits_few those of up to 8
// experts on v_mfma_f64_4x4x4f64; k_scored_choose adds the splits and does the rest with a wave or 16
// lanes a token.  Tokens go through both in chunks, which bounds the workspace.
#include <algorithm>
#include <type_traits>

#include "math_f64.h"

namespace moe {

namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

constexpr uint32_t kNowhere = 0x80000000u;  // past every array (below 2 GiB), also with some bytes added

// 8 columns of a token or of an expert, as stored.  A load takes a byte offset of the lane (kNowhere:
// zeros) and one of the wave, so that walking along d costs the vector ALU nothing: it and the fp64
// matrix instructions take turns.  inside: all of the wave's columns are below d.  widen: columns
// 4 h .. 4 h + 3 in fp64, exactly.
struct ChunkBf16 {  // d % 8 == 0
  typedef bf16_t Elem;
  uint4 v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t m, uint32_t lane_off, uint32_t wave_off,
                                       bool, int, int) {
    v = load16(m, lane_off, wave_off);
  }
  static __device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t m, uint32_t lane_off,
                                                 uint32_t wave_off) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(m, (int)lane_off, (int)wave_off, 0);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void widen(int h, double (&o)[4]) const {
    const uint32_t a = h ? v.z : v.x, b = h ? v.w : v.y;
    o[0] = __uint_as_float(a << 16);
    o[1] = __uint_as_float(a & 0xFFFF0000u);
    o[2] = __uint_as_float(b << 16);
    o[3] = __uint_as_float(b & 0xFFFF0000u);
  }
};
struct ChunkF32x4 {  // two 16-byte loads: d % 4 == 0, arrays on 4 bytes
  typedef float Elem;
  uint4 v[2];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t m, uint32_t lane_off, uint32_t wave_off,
                                       bool inside, int col, int d) {
    v[0] = ChunkBf16::load16(m, lane_off, wave_off);
    (void)inside;
    v[1] = ChunkBf16::load16(m, col + 4 < d ? lane_off + 16 : kNowhere, wave_off);
  }
  __device__ __forceinline__ void widen(int h, double (&o)[4]) const {
    o[0] = __uint_as_float(v[h].x);
    o[1] = __uint_as_float(v[h].y);
    o[2] = __uint_as_float(v[h].z);
    o[3] = __uint_as_float(v[h].w);
  }
};
struct ChunkF32 {  // any d: as ChunkF32x4 where all of the wave's columns are inside
  typedef float Elem;
  uint4 v[2];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t m, uint32_t lane_off, uint32_t wave_off,
                                       bool inside, int col, int d) {
    if (inside) {
      v[0] = ChunkBf16::load16(m, lane_off, wave_off);
      v[1] = ChunkBf16::load16(m, lane_off + 16, wave_off);
      return;
    }
    uint32_t w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      w[u] = __builtin_amdgcn_raw_buffer_load_b32(
          m, (int)(col + u < d ? lane_off + 4 * u : kNowhere), (int)wave_off, 0);
    v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    v[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ void widen(int h, double (&o)[4]) const {
    o[0] = __uint_as_float(v[h].x);
    o[1] = __uint_as_float(v[h].y);
    o[2] = __uint_as_float(v[h].z);
    o[3] = __uint_as_float(v[h].w);
  }
};

// ---------------------------------------------------------------- partial logits
// A block of WD waves takes 16 R tokens and 16 EBG experts: wave wd every (S WD)-th quad of 32 columns
// from quad split WD + wd on.  The waves are added in the order of wd, so equal calls give equal bits.
// Operands: lane l holds token or expert l % 16 and 8 consecutive columns, 8 (l / 16) of its quad on;
// instruction s multiplies column s of both, a permutation of the sum's order only.
// Bound from some thousand tokens on: the fp64 matrix instructions (64 cycles each, 73 TFLOP/s with
// nothing between) and the conversions, which they do not overlap with: T 65536, E 64, d 2048 281 us, 61
// TFLOP/s; accumulators in AGPRs would halve the rate.  Two rows of waves for 64 experts a block took as
// long, and 137 against 90 us for E 80 at T 16384, where they leave half of each last block idle.  W_r
// converted to fp64 by a launch ahead and read in the operands' order: 268 us at T 65536, but 73 + 5
// against 75 at T 16384.
template <typename Chunk, int R, int EBG, int WD>
__global__ __launch_bounds__(64 * WD) void k_scored_logits(
    const void* __restrict__ x, const void* __restrict__ w, int64_t T, int d, int E, int S,
    int64_t tok_base, int64_t n_tok, double* __restrict__ part) {
  constexpr int kPart = R * EBG * 256;
  __shared__ double lds[WD > 1 ? (WD - 1) * kPart : 1];
  const int lane = threadIdx.x & 63;
  const int wd = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  const int64_t tok0 = (int64_t)blockIdx.x * (16 * R);  // within the chunk
  const int e0 = (int)blockIdx.y * EBG * 16;
  const int split = blockIdx.z;
  constexpr uint32_t kSize = sizeof(typename Chunk::Elem);
  const int nq = (d + 31) / 32, stride = S * WD;
  const __amdgpu_buffer_rsrc_t xs = buffer_rsrc(x, (uint32_t)(T * d * kSize));
  const __amdgpu_buffer_rsrc_t ws = buffer_rsrc(w, (uint32_t)((int64_t)E * d * kSize));

  f64x4_t acc[R][EBG];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int b = 0; b < EBG; ++b) acc[r][b] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  Chunk xr[R], wr[EBG];
  uint32_t xo[R], wo[EBG];  // of the lane's columns in quad 0
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t t = tok0 + 16 * r + i;
    xo[r] = t < n_tok ? (uint32_t)((tok_base + t) * d + q * 8) * kSize : kNowhere;
  }
#pragma unroll
  for (int b = 0; b < EBG; ++b) {
    const int e = e0 + 16 * b + i;
    wo[b] = e < E ? (uint32_t)((int64_t)e * d + q * 8) * kSize : kNowhere;
  }
  // The wave's first NB tiles of experts: a tile that is past E is zeros.
  auto walk = [&](auto tiles) {
    constexpr int NB = decltype(tiles)::value;
    auto load = [&](int cq) {  // columns past d, and whole quads past the last, read as zeros
      const int col = cq * 32 + q * 8;
      // within the first row, and so within the array, whose size the lanes' offsets are held against
      const uint32_t at = cq < nq ? (uint32_t)cq * 32 * kSize : 0u;
#pragma unroll
      for (int r = 0; r < R; ++r)
        xr[r].load(xs, col < d ? xo[r] : kNowhere, at, cq * 32 + 32 <= d, col, d);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        wr[b].load(ws, col < d ? wo[b] : kNowhere, at, cq * 32 + 32 <= d, col, d);
    };
    int cq = split * WD + wd;
    load(cq);
    for (; cq < nq; cq += stride) {
      // half a chunk at a time: 16 registers of widened operands less
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        double xa[R][4], wb[NB][4];
#pragma unroll
        for (int r = 0; r < R; ++r) xr[r].widen(h, xa[r]);
#pragma unroll
        for (int b = 0; b < NB; ++b) wr[b].widen(h, wb[b]);
        if (h == 1) load(cq + stride);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b)
              acc[r][b] = __builtin_amdgcn_mfma_f64_16x16x4f64(xa[r][s], wb[b][s], acc[r][b], 0, 0, 0);
      }
    }
  };
  if (EBG == 1 || e0 + 16 < E)
    walk(std::integral_constant<int, EBG>{});
  else
    walk(std::integral_constant<int, 1>{});
  if constexpr (WD > 1) {
    if (wd > 0) {
      double* mine = lds + (wd - 1) * kPart;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int b = 0; b < EBG; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) mine[((r * EBG + b) * 4 + j) * 64 + lane] = acc[r][b][j];
    }
    __syncthreads();
    if (wd > 0) return;
#pragma unroll 1  // all waves' tiles at once would take the registers of a second block on the CU
    for (int o = 1; o < WD; ++o) {
      const double* other = lds + (o - 1) * kPart;
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

// ---------------------------------------------------------------- partial logits, up to 8 experts
// With 8 experts half of a 16 x 16 tile is empty.  v_mfma_f64_4x4x4f64 makes four 4 x 4 x 4 products: lane
// 16 g + 4 b + r holds row r of block b's A operand and column r of its B operand at step g, and
// receives row g, column r of its result.  The four blocks take four slices of 128 columns, so no two
// lanes load or convert the same values: lane (g, b, r) has 8 columns, 8 (4 b + g) on, of token 4 tg + r
// and of expert 4 eg + r.  A block of WD waves takes 16 tokens, wave wd every (S WD)-th 128 columns; the
// slices are added by lane moves, the waves in their order.  Whole calls against 16 x 16 tiles, us: E 8,
// T 32768, d 4096 67.8 / 87.7 (268 MB: 4.0 TB/s), T 16384, d 2048 22.9 / 26.7, T 64 no difference.
template <typename Chunk, int WD>
__global__ __launch_bounds__(64 * WD) void k_scored_logits_few(
    const void* __restrict__ x, const void* __restrict__ w, int64_t T, int d, int E, int S,
    int64_t tok_base, int64_t n_tok, double* __restrict__ part) {
  __shared__ double lds[WD - 1][8][64];
  const int lane = threadIdx.x & 63;
  const int wd = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, b = (lane >> 2) & 3, r = lane & 3;
  const int64_t tok0 = (int64_t)blockIdx.x * 16;  // within the chunk
  const int split = blockIdx.y;
  constexpr uint32_t kSize = sizeof(typename Chunk::Elem);
  const int nq = (d + 127) / 128, stride = S * WD;
  const __amdgpu_buffer_rsrc_t xs = buffer_rsrc(x, (uint32_t)(T * d * kSize));
  const __amdgpu_buffer_rsrc_t ws = buffer_rsrc(w, (uint32_t)((int64_t)E * d * kSize));
  double acc[4][2];
#pragma unroll
  for (int tg = 0; tg < 4; ++tg) acc[tg][0] = acc[tg][1] = 0.0;
  Chunk xr[4], wr[2];
  uint32_t xo[4], wo[2];
#pragma unroll
  for (int tg = 0; tg < 4; ++tg) {
    const int64_t t = tok0 + 4 * tg + r;
    xo[tg] = t < n_tok ? (uint32_t)((tok_base + t) * d + (4 * b + g) * 8) * kSize : kNowhere;
  }
#pragma unroll
  for (int eg = 0; eg < 2; ++eg)
    wo[eg] = 4 * eg + r < E ? (uint32_t)((int64_t)(4 * eg + r) * d + (4 * b + g) * 8) * kSize : kNowhere;
  auto load = [&](int cq) {
    const int col = cq * 128 + (4 * b + g) * 8;
    const bool inside = cq * 128 + 128 <= d;
    const uint32_t at = cq < nq ? (uint32_t)cq * 128 * kSize : 0u;  // within the first row
#pragma unroll
    for (int tg = 0; tg < 4; ++tg) xr[tg].load(xs, col < d ? xo[tg] : kNowhere, at, inside, col, d);
#pragma unroll
    for (int eg = 0; eg < 2; ++eg) wr[eg].load(ws, col < d ? wo[eg] : kNowhere, at, inside, col, d);
  };
  int cq = split * WD + wd;
  load(cq);
  for (; cq < nq; cq += stride) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      double xa[4][4], wb[2][4];
#pragma unroll
      for (int tg = 0; tg < 4; ++tg) xr[tg].widen(h, xa[tg]);
      wr[0].widen(h, wb[0]);
      wr[1].widen(h, wb[1]);
      if (h == 1) load(cq + stride);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int tg = 0; tg < 4; ++tg)
#pragma unroll
          for (int eg = 0; eg < 2; ++eg)
            acc[tg][eg] = __builtin_amdgcn_mfma_f64_4x4x4f64(xa[tg][s], wb[eg][s], acc[tg][eg], 0, 0, 0);
    }
  }
  auto moved = [](double v, int s) {
    return __longlong_as_double((long long)xor_partner((uint64_t)__double_as_longlong(v), s));
  };
#pragma unroll
  for (int tg = 0; tg < 4; ++tg)
#pragma unroll
    for (int eg = 0; eg < 2; ++eg) {
      acc[tg][eg] += moved(acc[tg][eg], 4);
      acc[tg][eg] += moved(acc[tg][eg], 8);
      if (wd > 0) lds[wd - 1][tg * 2 + eg][lane] = acc[tg][eg];
    }
  __syncthreads();
  if (wd > 0) return;
  double* out = part + (int64_t)split * n_tok * E;
  const int64_t t = tok0 + 4 * b + g;  // lane (g, b, r) stores token 4 b + g, experts r and 4 + r
#pragma unroll
  for (int eg = 0; eg < 2; ++eg) {
    double v = 0.0;
#pragma unroll
    for (int tg = 0; tg < 4; ++tg)
      if (tg == b) v = acc[tg][eg];
#pragma unroll
    for (int o = 1; o < WD; ++o) v += lds[o - 1][b * 2 + eg][lane];
    if (4 * eg + r < E && t < n_tok) out[t * E + 4 * eg + r] = v;
  }
}

// ---------------------------------------------------------------- scores and choice
constexpr int kMaxSplits = 8;

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

// The lanes that hold a token: 16 (a DPP row, see launch_choose) or the whole wave.  sum and max in a
// fixed order, every lane gets the result.
template <int LPT>
struct Lanes {
  // the lane move of dpp32, from whose zeros for lanes without a partner (there are none) the compiler
  // makes one instruction of a move and a maximum
  template <int CTRL>
  static __device__ __forceinline__ uint32_t moved(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
  }
  template <int CTRL>
  static __device__ __forceinline__ double moved(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)moved<CTRL>((uint32_t)(u >> 32)) << 32 |
                                            moved<CTRL>((uint32_t)u)));
  }
  static __device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)(
        ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane) << 32) |
        (uint32_t)__builtin_amdgcn_readlane((int)u, lane)));
  }
  // quads, then mirrored halves of a row and mirrored rows, then the wave's four rows
  template <typename Op>
  static __device__ __forceinline__ double all(double v, Op op) {
    v = op(v, moved<0xB1>(v));
    v = op(v, moved<0x4E>(v));
    v = op(v, moved<0x141>(v));
    v = op(v, moved<0x140>(v));
    if constexpr (LPT == 64)
      v = op(op(lane_of(v, 0), lane_of(v, 16)), op(lane_of(v, 32), lane_of(v, 48)));
    return v;
  }
  static __device__ __forceinline__ double sum(double v) {
    return all(v, [](double a, double b) { return a + b; });
  }
  static __device__ __forceinline__ double max(double v) {  // leaves NaN out
    return all(v, [](double a, double b) { return fmax(a, b); });
  }
  static __device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
    auto take = [&](uint32_t o) { v = o > v ? o : v; };
    take(moved<0xB1>(v));
    take(moved<0x4E>(v));
    take(moved<0x141>(v));
    take(moved<0x140>(v));
    return v;
  }
  // the largest key of the token's lanes, and the lowest lane (of LPT) that has it
  static __device__ __forceinline__ uint32_t best(uint32_t v, int& lane) {
    uint32_t m = row_max_u32(v);
    const int here = threadIdx.x & 63;
    if constexpr (LPT == 64) {
      const uint32_t a = __builtin_amdgcn_readlane(m, 0), b = __builtin_amdgcn_readlane(m, 16);
      const uint32_t c = __builtin_amdgcn_readlane(m, 32), d = __builtin_amdgcn_readlane(m, 48);
      const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
      m = ab > cd ? ab : cd;
      lane = __ffsll((long long)__ballot(v == m)) - 1;
    } else {
      const uint64_t row = __ballot(v == m) >> (here & 48);
      lane = __ffs((int)(row & 0xFFFFu)) - 1;
    }
    return m;
  }
};

// The two largest keys of two pairs (best >= second).
__device__ __forceinline__ void two_largest(uint32_t& best, uint32_t& second, uint32_t b2, uint32_t s2) {
  const uint32_t low = best < b2 ? best : b2, high = second > s2 ? second : s2;
  best = best > b2 ? best : b2;
  second = low > high ? low : high;
}
// one expert that is on speaks for its group alone; a group without any is the last
__device__ __forceinline__ uint32_t group_key(uint32_t best, uint32_t second, int top2) {
  return top2 && second ? order_key(key_value(best) + key_value(second)) : best;
}

// LPT lanes a token, lane l of them holds experts l NV .. l NV + NV - 1, so that the lowest expert of
// equal ones is the lowest lane's first.  Groups that are a power of two of a wave's lanes are
// reduced by lane moves, others through LDS ([tokens of the block][E + n_groups] keys).
template <int LPT, int NV>
__global__ __launch_bounds__(256) void k_scored_choose(const ChooseArgs a) {
  using W = Lanes<LPT>;
  constexpr int TPB = 256 / LPT;
  extern __shared__ uint32_t shared_keys[];
  const int l = threadIdx.x % LPT, row = threadIdx.x / LPT;
  const int64_t t = (int64_t)blockIdx.x * TPB + row;
  const bool there = t < a.n_tok;
  const int64_t tt = a.tok_base + t;
  const bool real = there && (!a.mask || a.mask[tt]);
  const int E = a.E, k = a.k, e0 = l * NV;
  const int lanes = (E + NV - 1) / NV;  // that hold experts

  // Loads past E or the tokens take the last expert's or the first token's in their place, and need no
  // branch that would have to be waited for.
  double z[NV];
  float sb[NV];
  const double* part = a.part + (there ? t * E : 0);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = e0 + i < E ? e0 + i : E - 1;
    z[i] = part[e];
    sb[i] = a.score_bias ? a.score_bias[e] : 0.0f;
  }
  float rb[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) rb[i] = a.b_router ? a.b_router[e0 + i < E ? e0 + i : E - 1] : 0.0f;
  if (a.S > 1) {
    // all splits' loads before the first sum: the compiler on its own waits for one after the other
    double v[kMaxSplits - 1][NV];
#pragma unroll
    for (int s = 1; s < kMaxSplits; ++s) {
      const double* from = part + (s < a.S ? (int64_t)s * a.n_tok * E : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) v[s - 1][i] = from[e0 + i < E ? e0 + i : E - 1];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 1; s < kMaxSplits; ++s)
#pragma unroll
      for (int i = 0; i < NV; ++i) z[i] += s < a.S ? v[s - 1][i] : 0.0;
  }
  if (a.b_router)
#pragma unroll
    for (int i = 0; i < NV; ++i) z[i] += (double)rb[i];
  if (there && a.logits)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < E) a.logits[tt * E + e0 + i] = real ? (float)z[i] : 0.0f;

  // scores: e^-l gives 1 / (1 + e^-l), e^(l - m) its share of the sum; 0 past E
  double m = 0.0;
  if (!a.sigmoid) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < E) m = fmax(m, z[i]);
    m = W::max(m);
    if (m == -INFINITY) m = 0.0;  // nothing but -inf (and NaN, which fmax leaves out): zeros
  }
  double p[NV], sum = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    p[i] = e0 + i < E ? exp_clamped(a.sigmoid ? -z[i] : z[i] - m) : 0.0;
    sum += p[i];
  }
  double inv = 1.0;
  if (!a.sigmoid) {
    sum = W::sum(sum);
    inv = 1.0 / (sum == 0.0 ? 1.0 : sum);
  }
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    p[i] = a.sigmoid ? reciprocal(1.0 + p[i]) : p[i] * inv;
    const bool on = e0 + i < E && sb[i] != -INFINITY;
    // the bias is added also where there is none: a score is no -0
    key[i] = on ? order_key((float)p[i] + sb[i]) : 0u;
  }

  if (a.topk_groups < a.n_groups) {  // uniform over the grid
    const int G = a.n_groups, gs = E / G, lpg = gs / NV;  // lanes a group
    if (LPT == 64 && lpg * NV == gs && (lpg & (lpg - 1)) == 0) {
      uint32_t best = 0, second = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) two_largest(best, second, key[i], 0u);
#pragma unroll
      for (int s = 1; s < 64; s <<= 1)
        if (s < lpg) {
          const uint64_t o = xor_partner(((uint64_t)best << 32) | second, s);
          two_largest(best, second, (uint32_t)(o >> 32), (uint32_t)o);
        }
      const uint32_t mine = group_key(best, second, a.top2);
      // a group stays if fewer than topk_groups are better (or as good and before it)
      const int g = l / lpg;
      int better = 0;
      for (int o = 0; o < G; ++o) {
        const uint32_t other = __builtin_amdgcn_readlane(mine, o * lpg);
        better += other > mine || (other == mine && o < g);
      }
      if (better >= a.topk_groups)
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = 0;
    } else {
      uint32_t* keys = shared_keys + row * (E + G);
      uint32_t* group = keys + E;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (e0 + i < E) keys[e0 + i] = key[i];
      __syncthreads();
      for (int g = l; g < G; g += LPT) {
        uint32_t best = 0, second = 0;
        for (int j = 0; j < gs; ++j) two_largest(best, second, keys[g * gs + j], 0u);
        group[g] = group_key(best, second, a.top2);
      }
      __syncthreads();
      for (int g = l; g < G; g += LPT) {
        const uint32_t mine = group[g];
        int better = 0;
        for (int o = 0; o < G; ++o) better += group[o] > mine || (group[o] == mine && o < g);
        keys[g] = better < a.topk_groups;  // the experts' keys are in registers
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (e0 + i < E && !keys[(e0 + i) / gs]) key[i] = 0;
    }
  }

  int taken = 0;
  if (real)
    for (; taken < k; ++taken) {
      uint32_t best = key[0], at = 0;
#pragma unroll
      for (int i = 1; i < NV; ++i)
        if (key[i] > best) {
          best = key[i];
          at = i;
        }
      int lane;
      if (W::best(l < lanes ? best : 0u, lane) < kLeastKey) break;  // all lanes of the token agree
      if (l == lane)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (at == (uint32_t)i) key[i] = 1 + taken;
    }
  if (!there) return;

  auto chosen = [&](int i) { return key[i] != 0 && key[i] < kLeastKey; };
  double total = 1.0;
  if (a.renormalize) {
    total = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (chosen(i)) total += p[i];
    total = W::sum(total);
    // Scores near the end of fp64's range or below it: e^l instead, from the largest chosen logit (1 + e^l
    // is 1 there); all of them zero (-inf): the gates are zero.  From 1e-200 on, what the range takes of
    // a smaller score reaches no gate: exp_clamped's floor (1e-304) and denormal numbers (below 1e-307)
    // are 1e-104 of the sum at most, which times the largest scale (3.4e38) is nothing in fp32; and
    // scale / total stays finite.
    if (total < 1e-200) {
      m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (chosen(i)) m = fmax(m, z[i]);
      m = W::max(m);
      if (m == -INFINITY) m = 0.0;
      total = 0.0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (chosen(i)) {
          p[i] = exp_clamped(z[i] - m);
          total += p[i];
        }
      total = W::sum(total);
      if (total == 0.0) total = 1.0;
    }
  }
  const double factor = a.scale / total;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (chosen(i)) {
      const int64_t at = tt * k + (key[i] - 1);
      a.ids[at] = e0 + i;
      a.gates[at] = (float)(p[i] * factor);
    }
  for (int c = taken + l; c < k; c += LPT) {  // masked, or too few experts are on
    a.ids[tt * k + c] = -1;
    a.gates[tt * k + c] = 0.0f;
  }
}

// ---------------------------------------------------------------- launches
struct Plan {
  int64_t chunk;  // tokens that go through the two launches at a time
  int S;          // splits of the columns
  bool few;       // up to 8 experts
  bool large;     // blocks of 32 tokens x 32 (16) experts instead of 16 x 16
};

constexpr int64_t kPartBytes = (int64_t)64 << 20;  // of partial logits at most
int most_splits(int d, int columns) { return (d + columns - 1) / columns; }

// Large tiles convert each value for two products, and conversions and fp64 products take turns (12
// and 64 cycles); small tiles and split columns spread more evenly over the CUs.  The least of
//   (16 x 16 tiles on the CU with most) * (columns of a block) * (us a tile and column)
// with 15 % more where that is one block alone, 2 us for the longer start and end of a large block, and
// the partial logits of each split, written and read.  us measured, large tiles and small ones with
// the splits in brackets, bf16, d 2048: T 16384, E 64 74 (1) and 84 (1); T 16400 89 (1), 78 (3) and 86 (1);
// T 2048, E 160 37 (1), 28 (4) and 27 (1); T 4096, E 160 55 (1), 48 (2) and 53 (1); T 250, E 64 21 (1),
// 8.2 (4) and 8.9 (1), 4.4 (4).
Plan plan(const moe_shape& s) {
  constexpr int kCUs = 256;
  Plan p{0, 1, s.n_experts <= 8, false};
  const int64_t tokens16 = (s.T + 15) / 16, tokens32 = (s.T + 31) / 32;
  if (p.few) {  // at least 128 columns for each of 4 waves
    const int64_t most = most_splits(s.d_model, 512);
    p.S = (int)std::max<int64_t>(1, std::min<int64_t>({512 / std::max<int64_t>(tokens16, 1), most, kMaxSplits}));
  } else {
    const int quads = (s.d_model + 31) / 32, E16 = (s.n_experts + 15) / 16;
    const double split_us = 0.1 + (double)(s.T * s.n_experts * 8) * 1e-7;
    double least = INFINITY;
    for (int large = 0; large < 2; ++large) {
      const int waves = large ? 4 : 8;
      const double us = !large ? 2.45e-3 : E16 == 1 ? 2.3e-3 : 2.15e-3;
      const int most = std::min(most_splits(s.d_model, 32 * waves), kMaxSplits);
      for (int S = 1; S <= most; ++S) {
        if (S > 1 && tokens32 * 32 * s.n_experts * 8 * S > kPartBytes) break;  // one part of tokens
        int64_t tiles, block = 1;  // on the CU with most, and in a block
        if (!large) {
          tiles = (tokens16 * E16 * S + kCUs - 1) / kCUs;
        } else if (E16 % 2 == 0) {
          block = 4;
          tiles = 4 * ((tokens32 * (E16 / 2) * S + kCUs - 1) / kCUs);
        } else {  // the last block of each 32 tokens has half the experts
          block = E16 > 1 ? 4 : 2;
          tiles = std::max<int64_t>(block, 2 * ((tokens32 * E16 * S + kCUs - 1) / kCUs));
        }
        const int columns = 32 * waves * ((quads + S * waves - 1) / (S * waves));
        const double cost = (double)tiles * columns * us * (tiles == block ? 1.15 : 1.0) +
                            (S - 1) * split_us + (large ? 2.0 : 0.0);
        if (cost < least) least = cost, p.S = S, p.large = large != 0;
      }
    }
  }
  p.chunk = std::min<int64_t>(s.T, kPartBytes / (8 * s.n_experts * p.S) / 32 * 32);
  return p;
}

template <typename Chunk, int R, int EBG, int WD>
hipError_t launch_logits(const moe_shape& s, const void* x, const void* w, const Plan& p,
                         int64_t base, int64_t n, double* part, hipStream_t st) {
  const dim3 grid((unsigned)((n + 16 * R - 1) / (16 * R)),
                  (unsigned)((s.n_experts + 16 * EBG - 1) / (16 * EBG)), (unsigned)p.S);
  hipLaunchKernelGGL((k_scored_logits<Chunk, R, EBG, WD>), grid, dim3(64 * WD), 0, st, x, w,
                     s.T, s.d_model, s.n_experts, p.S, base, n, part);
  return hipGetLastError();
}

template <typename Chunk>
hipError_t logits_any(const moe_shape& s, const void* x, const void* w, const Plan& p, int64_t base,
                      int64_t n, double* part, hipStream_t st) {
  if (p.few) {
    constexpr int WD = 4;
    hipLaunchKernelGGL((k_scored_logits_few<Chunk, WD>), dim3((unsigned)((n + 15) / 16), (unsigned)p.S),
                       dim3(64 * WD), 0, st, x, w, s.T, s.d_model, s.n_experts, p.S, base, n, part);
    return hipGetLastError();
  }
  if (!p.large) return launch_logits<Chunk, 1, 1, 8>(s, x, w, p, base, n, part, st);
  if (s.n_experts <= 16) return launch_logits<Chunk, 2, 1, 4>(s, x, w, p, base, n, part, st);
  return launch_logits<Chunk, 2, 2, 4>(s, x, w, p, base, n, part, st);
}

hipError_t launch_choose(const ChooseArgs& a, hipStream_t st) {
  auto go = [&](auto kern, int tokens) {
    const size_t lds = a.topk_groups < a.n_groups ? (size_t)tokens * 4 * (a.E + a.n_groups) : 0;
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.n_tok + tokens - 1) / tokens)), dim3(256), lds, st, a);
    return hipGetLastError();
  };
  if (a.E <= 16) return go(k_scored_choose<16, 1>, 16);
  if (a.E <= 32) return go(k_scored_choose<16, 2>, 16);
  // A wave a token is sooner done, 16 lanes take fewer instructions.  us, wave / 16 lanes: E 64, T 64
  // 3.9 / 4.8, 4096 4.5 / 5.2, 16384 10.3 / 9.9 (with 8 groups 13.5 / 11.9); E 40, top-8, T 65536 42.2
  // / 25.5.  Above 64 experts 16 lanes hold too many each: E 128, T 16384 14.4 / 24.4.
  if (a.E <= 64 && a.n_tok >= 8192) return go(k_scored_choose<16, 4>, 16);
  if (a.E <= 64) return go(k_scored_choose<64, 1>, 4);
  if (a.E <= 128) return go(k_scored_choose<64, 2>, 4);
  return go(k_scored_choose<64, 4>, 4);
}

}  // namespace

// For as many splits as the columns allow, so that no smaller batch of the same kind takes more.
size_t route_scored_ws_bytes(const moe_shape& s) {
  const int most = std::min(most_splits(s.d_model, s.n_experts <= 8 ? 512 : 128), kMaxSplits);
  return ((size_t)std::min<int64_t>(kPartBytes, s.T * s.n_experts * 8 * most) + 255) & ~(size_t)255;
}

hipError_t launch_route_scored(const moe_shape& s, const moe_routing& r, const void* x,
                               const void* w_router, const float* b_router,
                               const float* score_bias, const uint8_t* mask, int32_t* ids,
                               float* gates, float* logits, void* ws, hipStream_t st) {
  const Plan p = plan(s);
  double* part = (double*)ws;
  for (int64_t base = 0; base < s.T; base += p.chunk) {
    const int64_t n = s.T - base < p.chunk ? s.T - base : p.chunk;
    hipError_t err =
        s.dtype == MOE_BF16    ? logits_any<ChunkBf16>(s, x, w_router, p, base, n, part, st)
        : s.d_model % 4 == 0 ? logits_any<ChunkF32x4>(s, x, w_router, p, base, n, part, st)
                             : logits_any<ChunkF32>(s, x, w_router, p, base, n, part, st);
    if (err != hipSuccess) return err;
    ChooseArgs a{part, p.S, base, n, s.n_experts, s.top_k, r.score == MOE_SCORE_SIGMOID,
                 r.n_groups, r.topk_groups, r.group_score == MOE_GROUP_TOP_TWO, r.renormalize,
                 (double)r.scale, b_router, score_bias, mask, ids, gates, logits};
    if ((err = launch_choose(a, st)) != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
