// Expert FFN on 4-bit weights: the two grouped products over the routed rows.
//
//   H[s, n] = act(sum_k x[row_token[s], k] W1[e, n, k] + b1[e, n]),  Y[s, n] = sum_k H[s, k] W2[e, n, k] + b2[e, n]
// with W[n, k] = scale[n, k / group] value(code[n, k]) (quantize.hip has the storage).  For every
// group, v_mfma_f32_16x16x32_bf16 sums x value(code), both exact in bf16, in fp32, and the scale
// multiplies that sum once, in fp32: no weight is rounded.  H is stored as bf16, as the bf16
// layer stores it.
//
// Roles: token rows are the A operand (lane n: row n of 16, 8 K values from 8 (lane / 16)), weight
// rows the B operand, so a lane holds one feature's results for four token rows and one scale
// serves all four.
#include "moe_internal.h"

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kQNone = 0;   // Y = acc + bias
constexpr int kQSilu = 1;   // H = SiLU(acc + bias)
constexpr int kQGated = 2;  // H = SiLU(gate) * up, no bias

__device__ __forceinline__ bf16x8_t qfrag(uint4 v) { return __builtin_bit_cast(bf16x8_t, v); }

// the eight values of a dword of codes, as a fragment
__device__ __forceinline__ bf16x8_t values_of(uint32_t c) {
  uint4 v;
  v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0));
  v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1));
  v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2));
  v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3));
  return qfrag(v);
}

__device__ __forceinline__ float silu(float v) {
  return v / (1.0f + __builtin_amdgcn_exp2f(-1.44269504f * v));
}

// The scales of one row for one block of 128 columns (128 / GROUP bf16).
template <int GROUP>
struct Scales {
  static constexpr int N = 128 / GROUP;
  uint32_t w[(N + 1) / 2];
  __device__ __forceinline__ void load(const bf16_t* p) {
    if constexpr (N == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    } else if constexpr (N == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *p;
    }
  }
  __device__ __forceinline__ float get(int g) const {
    return __uint_as_float(g % 2 ? w[g / 2] & 0xFFFF0000u : w[g / 2] << 16);
  }
};

struct QArgs {
  const bf16_t* A;           // token rows [a_rows, K]
  const int32_t* row_token;  // row of A of each slot, or NULL: the slot itself
  const int32_t* offsets;    // [E + 1]
  const uint4* codes;
  const bf16_t* scales;
  const bf16_t* bias;  // [E, N] or NULL
  bf16_t* out;         // [slots, N]
  int E, N, K;         // N output features (a gated expert has 2 N weight rows)
  int64_t a_rows;
  int out_rows;  // rows of out: no slot at or past it is computed
};

// Expert number `want` (from 0) among those with rows, or -1; wave-uniform, all lanes call.
__device__ __forceinline__ int nth_active(const int32_t* __restrict__ offsets, int E, int want) {
  const int lane = threadIdx.x & 63;
  int seen = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    uint64_t m = __ballot(e < E && offsets[e + 1] > offsets[e]);
    const int here = __popcll(m);
    if (want < seen + here) {
      for (int i = want - seen; i > 0; --i) m &= m - 1;
      return e0 + __ffsll((long long)m) - 1;
    }
    seen += here;
  }
  return -1;
}

// ---------------------------------------------------------------- few rows an expert
// A block takes 16 FT weight rows of one expert and all of its token rows, 16 RT at a time; its WK
// waves take the 128-column blocks of K in turn, and their sums are added in LDS, in wave order.
// Weights go from HBM to registers, PF blocks ahead, each 16-byte load feeding four matrix
// instructions; the token rows come from L2.
template <int RT, int FT, int WK, int GROUP, int ACT>
__global__ __launch_bounds__(64 * WK) void k_quant_rows(QArgs a) {
  constexpr int PF = 2;
  constexpr bool GATED = ACT == kQGated;
  constexpr int FO = GATED ? FT / 2 : FT;  // output tiles
  static_assert(!GATED || FT % 2 == 0, "gate and up tiles in pairs");
  __shared__ f32x4_t red[WK][RT * FT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  const int e = nth_active(a.offsets, a.E, blockIdx.y);
  if (e < 0) return;  // block-uniform
  const int row0 = a.offsets[e], rows = min(a.offsets[e + 1], a.out_rows) - row0;
  const int KC = (a.K + 127) / 128;
  const int wrows = GATED ? 2 * a.N : a.N;  // weight rows of the expert (a multiple of 8)
  const int f0 = blockIdx.x * FO * 16;
  // weight row of lane n in tile f, clamped (the results of clamped lanes are not stored)
  const uint4* cp[FT];
  const bf16_t* sp[FT];
#pragma unroll
  for (int f = 0; f < FT; ++f) {
    int r = f0 + (f % FO) * 16 + n;
    r = r < a.N ? r : a.N - 8 + (n & 7);
    if (GATED && f >= FO) r += a.N;
    const int64_t row = (int64_t)e * wrows + r;
    cp[f] = a.codes + row / 8 * KC * 32 + kg * 8 + r % 8;
    sp[f] = a.scales + row * KC * (128 / GROUP);
  }
  for (int r0 = 0; r0 < rows; r0 += 16 * RT) {
    const bf16_t* xp[RT];
    bool in[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = r0 + rt * 16 + n;
      int64_t at = -1;
      if (r < rows) at = a.row_token ? a.row_token[row0 + r] : row0 + r;
      in[rt] = at >= 0 && at < a.a_rows;
      xp[rt] = a.A + (in[rt] ? at : 0) * a.K + kg * 8;
    }
    f32x4_t acc[RT][FT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int f = 0; f < FT; ++f) acc[rt][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    uint4 cw[PF][FT], xw[PF][RT][4];
    Scales<GROUP> sc[PF][FT];
    auto load = [&](int p, int kc) {
      if (kc >= KC) return;
#pragma unroll
      for (int f = 0; f < FT; ++f) {
        cw[p][f] = cp[f][(int64_t)kc * 32];
        sc[p][f].load(sp[f] + kc * (128 / GROUP));
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = kc * 128 + j * 32;
          xw[p][rt][j] = make_uint4(0, 0, 0, 0);
          if (in[rt] && k + kg * 8 < a.K) xw[p][rt][j] = *reinterpret_cast<const uint4*>(xp[rt] + k);
        }
    };
#pragma unroll
    for (int p = 0; p < PF; ++p) load(p, wave + p * WK);
    for (int kc = wave; kc < KC; kc += PF * WK) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        if (kc + p * WK >= KC) break;
#pragma unroll
        for (int f = 0; f < FT; ++f) {
          const uint32_t c[4] = {cw[p][f].x, cw[p][f].y, cw[p][f].z, cw[p][f].w};
#pragma unroll
          for (int g = 0; g < 128 / GROUP; ++g) {
            const float s = sc[p][f].get(g);
            f32x4_t t[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) t[rt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = g * (GROUP / 32); j < (g + 1) * (GROUP / 32); ++j) {
              const bf16x8_t B = values_of(c[j]);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt)
                t[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qfrag(xw[p][rt][j]), B, t[rt], 0, 0, 0);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[rt][f][i] = fmaf(s, t[rt][i], acc[rt][f][i]);
          }
        }
        load(p, kc + (p + PF) * WK);
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int f = 0; f < FT; ++f) red[wave][rt * FT + f][lane] = acc[rt][f];
    __syncthreads();
    for (int i = threadIdx.x; i < RT * FO * 64; i += 64 * WK) {
      const int rt = i / (FO * 64), f = i / 64 % FO, ln = i % 64;
      f32x4_t v = red[0][rt * FT + f][ln];
      for (int w = 1; w < WK; ++w) v += red[w][rt * FT + f][ln];
      const int feat = f0 + f * 16 + ln % 16;
      if (feat >= a.N) continue;
      if constexpr (GATED) {
        f32x4_t u = red[0][rt * FT + FO + f][ln];
        for (int w = 1; w < WK; ++w) u += red[w][rt * FT + FO + f][ln];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = silu(v[j]) * u[j];
      } else {
        const float b = a.bias ? bf16_to_f32(a.bias[(int64_t)e * a.N + feat]) : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = ACT == kQSilu ? silu(v[j] + b) : v[j] + b;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + rt * 16 + ln / 16 * 4 + j;
        if (r < rows) a.out[(int64_t)(row0 + r) * a.N + feat] = (bf16_t)pack_bf16x2(v[j], 0.0f);
      }
    }
    __syncthreads();  // red is written again by the next rows
  }
}

// ---------------------------------------------------------------- many rows an expert
// A block takes 16 RT token rows x 256 weight rows (four waves of 64).  A block of 128 columns of
// the token rows goes through LDS in fragment order (16 lanes a row group, 1 KiB a fragment), so
// the four waves read it without conflicts; each wave converts its own weights, once for all
// token rows.
template <int RT, int GROUP, int ACT>
__global__ __launch_bounds__(256) void k_quant_tiles(QArgs a) {
  constexpr bool GATED = ACT == kQGated;
  constexpr int FT = 4, FO = GATED ? 2 : 4;
  constexpr int TM = 16 * RT;
  __shared__ uint4 xs[2][RT * 4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  // token tile `mt` of all experts' tiles
  constexpr int NB = GATED ? 128 : 256;
  const int NT = (a.N + NB - 1) / NB;
  const int mt = blockIdx.x / NT, nt = blockIdx.x % NT;
  int e = -1, row0 = 0, rows = 0;
  {
    int seen = 0;
    for (int i = 0; i < a.E; ++i) {
      const int lo = a.offsets[i], hi = min(a.offsets[i + 1], a.out_rows);
      const int t = (hi - lo + TM - 1) / TM;
      if (mt < seen + t) {
        e = i;
        row0 = lo + (mt - seen) * TM;
        rows = hi - row0 < TM ? hi - row0 : TM;
        break;
      }
      seen += t;
    }
  }
  if (e < 0) return;  // block-uniform
  const int KC = (a.K + 127) / 128;
  const int wrows = GATED ? 2 * a.N : a.N;
  const int f0 = (nt * 4 + wave) * FO * 16;
  const uint4* cp[FT];
  const bf16_t* sp[FT];
#pragma unroll
  for (int f = 0; f < FT; ++f) {
    int r = f0 + (f % FO) * 16 + n;
    r = r < a.N ? r : a.N - 8 + (n & 7);
    if (GATED && f >= FO) r += a.N;
    const int64_t row = (int64_t)e * wrows + r;
    cp[f] = a.codes + row / 8 * KC * 32 + kg * 8 + r % 8;
    sp[f] = a.scales + row * KC * (128 / GROUP);
  }
  // this thread's share of the staging: fragments (rt, j = wave), lane (n, kg)
  const bf16_t* xp[RT];
  bool in[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = rt * 16 + n;
    int64_t at = -1;
    if (r < rows) at = a.row_token ? a.row_token[row0 + r] : row0 + r;
    in[rt] = at >= 0 && at < a.a_rows;
    xp[rt] = a.A + (in[rt] ? at : 0) * a.K + wave * 32 + kg * 8;
  }
  uint4 xr[RT], cw[FT];
  Scales<GROUP> sc[FT];
  auto load_x = [&](int kc) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      xr[rt] = make_uint4(0, 0, 0, 0);
      if (in[rt] && kc * 128 + wave * 32 + kg * 8 < a.K)
        xr[rt] = *reinterpret_cast<const uint4*>(xp[rt] + kc * 128);
    }
  };
  auto load_w = [&](int kc) {
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      cw[f] = cp[f][(int64_t)kc * 32];
      sc[f].load(sp[f] + kc * (128 / GROUP));
    }
  };
  f32x4_t acc[RT][FT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int f = 0; f < FT; ++f) acc[rt][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  load_x(0);
  load_w(0);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) xs[0][rt * 4 + wave][lane] = xr[rt];
  __syncthreads();
  for (int kc = 0; kc < KC; ++kc) {
    bf16x8_t B[FT][4];
    float s[FT][128 / GROUP];
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      B[f][0] = values_of(cw[f].x);
      B[f][1] = values_of(cw[f].y);
      B[f][2] = values_of(cw[f].z);
      B[f][3] = values_of(cw[f].w);
#pragma unroll
      for (int g = 0; g < 128 / GROUP; ++g) s[f][g] = sc[f].get(g);
    }
    const bool more = kc + 1 < KC;
    if (more) {
      load_x(kc + 1);
      load_w(kc + 1);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      bf16x8_t A[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) A[j] = qfrag(xs[kc & 1][rt * 4 + j][lane]);
#pragma unroll
      for (int g = 0; g < 128 / GROUP; ++g) {
        f32x4_t t[FT];
#pragma unroll
        for (int f = 0; f < FT; ++f) t[f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = g * (GROUP / 32); j < (g + 1) * (GROUP / 32); ++j)
#pragma unroll
          for (int f = 0; f < FT; ++f)
            t[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[j], B[f][j], t[f], 0, 0, 0);
#pragma unroll
        for (int f = 0; f < FT; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][f][i] = fmaf(s[f][g], t[f][i], acc[rt][f][i]);
      }
    }
    if (more) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) xs[(kc + 1) & 1][rt * 4 + wave][lane] = xr[rt];
    }
    __syncthreads();
  }
#pragma unroll
  for (int f = 0; f < FO; ++f) {
    const int feat = f0 + f * 16 + n;
    if (feat >= a.N) continue;
    const float b = !GATED && a.bias ? bf16_to_f32(a.bias[(int64_t)e * a.N + feat]) : 0.0f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = rt * 16 + kg * 4 + j;
        float v = acc[rt][f][j];
        if constexpr (GATED)
          v = silu(v) * acc[rt][FO + f][j];
        else
          v = ACT == kQSilu ? silu(v + b) : v + b;
        if (r < rows) a.out[(int64_t)(row0 + r) * a.N + feat] = (bf16_t)pack_bf16x2(v, 0.0f);
      }
  }
}

template <int GROUP, int ACT>
hipError_t run_quant(const QArgs& a, int64_t rows_ub, int64_t mean_rows, hipStream_t st) {
  constexpr bool GATED = ACT == kQGated;
  const int64_t active = rows_ub < a.E ? rows_ub : a.E;
  if (mean_rows > 64) {
    constexpr int NB = GATED ? 128 : 256;
    const int64_t tiles = (rows_ub + 127) / 128 + a.E;
    return launch_timed(k_quant_tiles<8, GROUP, ACT>,
                        dim3((unsigned)((a.N + NB - 1) / NB * tiles)), dim3(256), 0, st, a);
  }
  auto grid = [&](int FT) {
    const int cols = 16 * (GATED ? FT / 2 : FT);
    return dim3((unsigned)((a.N + cols - 1) / cols), (unsigned)active);
  };
  if (mean_rows > 24)
    return launch_timed(k_quant_rows<4, 2, 8, GROUP, ACT>, grid(2), dim3(512), 0, st, a);
  if (mean_rows > 8)
    return launch_timed(k_quant_rows<2, 4, 8, GROUP, ACT>, grid(4), dim3(512), 0, st, a);
  return launch_timed(k_quant_rows<1, 4, 8, GROUP, ACT>, grid(4), dim3(512), 0, st, a);
}

template <int ACT>
hipError_t run_quant(int group, const QArgs& a, int64_t rows_ub, int64_t mean_rows,
                     hipStream_t st) {
  if (rows_ub <= 0) return hipSuccess;
  if (group == 32) return run_quant<32, ACT>(a, rows_ub, mean_rows, st);
  if (group == 64) return run_quant<64, ACT>(a, rows_ub, mean_rows, st);
  return run_quant<128, ACT>(a, rows_ub, mean_rows, st);
}

}  // namespace

hipError_t launch_quant_up(const moe_shape& s, const moe_quantized_experts& q, const void* x,
                           const int32_t* row_token, const int32_t* offsets, void* h,
                           int64_t rows_ub, hipStream_t st) {
  QArgs a = {(const bf16_t*)x,
             row_token,
             offsets,
             (const uint4*)q.w1_codes,
             (const bf16_t*)q.w1_scales,
             q.gated ? nullptr : (const bf16_t*)q.b1,
             (bf16_t*)h,
             s.n_experts,
             s.d_ff,
             s.d_model,
             s.T,
             (int)rows_ub};
  const int64_t mean = (rows_ub + s.n_experts - 1) / s.n_experts;
  return q.gated ? run_quant<kQGated>(q.group, a, rows_ub, mean, st)
                 : run_quant<kQSilu>(q.group, a, rows_ub, mean, st);
}

hipError_t launch_quant_down(const moe_shape& s, const moe_quantized_experts& q, const void* h,
                             const int32_t* offsets, void* y, int64_t rows_ub, hipStream_t st) {
  QArgs a = {(const bf16_t*)h,
             nullptr,
             offsets,
             (const uint4*)q.w2_codes,
             (const bf16_t*)q.w2_scales,
             q.gated ? nullptr : (const bf16_t*)q.b2,
             (bf16_t*)y,
             s.n_experts,
             s.d_model,
             s.d_ff,
             rows_ub,
             (int)rows_ub};
  const int64_t mean = (rows_ub + s.n_experts - 1) / s.n_experts;
  return run_quant<kQNone>(q.group, a, rows_ub, mean, st);
}

}  // namespace moe
