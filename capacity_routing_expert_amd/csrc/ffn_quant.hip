// Expert FFN on 4-bit weights: the two grouped products over the routed rows.
//
//   H[s, n] = act(sum_k x[row_token[s], k] W1[e, n, k] + b1[e, n])
//   Y[s, n] = sum_k H[s, k] W2[e, n, k] + b2[e, n]
// with W[n, k] = scale[n, k / group] value(code[n, k]) (quantize.hip has the storage).  For every
// group, v_mfma_f32_16x16x32_bf16 sums x value(code), both exact in bf16, in fp32, and the scale
// multiplies that sum once, in fp32: no weight is rounded.  H is stored as bf16, as the bf16
// layer stores it.
//
// Roles: token rows are the A operand (lane n: row n of 16, 8 K values from 8 (lane / 16)), weight
// rows the B operand, so a lane holds one feature's results for four token rows and one scale
// serves all four.  A 16-byte load of codes feeds a lane's part of four matrix instructions (128
// columns), and the waves of a block read neighbouring rows of the same column block: runs of
// 4 to 16 KiB.  The token rows go through LDS in fragment order (1 KiB a fragment, read without
// conflicts), loaded once for all waves of a block.
//
// Everything that a buffer descriptor is made of is wave-uniform and kept scalar (readfirstlane):
// the loads then need no loop over descriptor values.
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
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (N == 4) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
      w[0] = v[0];
      w[1] = v[1];
    } else if constexpr (N == 2) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
    } else {
      w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
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
  int xcds;      // XCDs that share one row tile's feature tiles: 2 or 8
  int out_rows;  // rows of out: no slot at or past it is computed
};

// Row tile `want` of TM rows, counted over the experts: its expert and rows; false past the last.
// Lane l adds up the tiles of experts 4 l .. 4 l + 3, a prefix sum over the lanes finds the owner.
// The results are scalars.
template <int TM>
__device__ __forceinline__ bool row_tile(const QArgs& a, int want, int& e, int& row0, int& rows) {
  const int lane = threadIdx.x & 63;
  int te[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = lane * 4 + j;
    const int n = i < a.E ? min(a.offsets[i + 1], a.out_rows) - a.offsets[i] : 0;
    te[j] = n > 0 ? (n + TM - 1) / TM : 0;
    sum += te[j];
  }
  int inc = sum;
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o, 64);
    if (lane >= o) inc += v;
  }
  if (want >= __builtin_amdgcn_readfirstlane(__shfl(inc, 63, 64))) return false;
  const int owner = __builtin_amdgcn_readfirstlane(__ffsll((long long)__ballot(want < inc)) - 1);
  int run = inc - sum, ex = lane * 4, at = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (want >= run && want < run + te[j]) {
      ex = lane * 4 + j;
      at = want - run;
    }
    run += te[j];
  }
  e = __builtin_amdgcn_readfirstlane(__shfl(ex, owner, 64));
  at = __builtin_amdgcn_readfirstlane(__shfl(at, owner, 64));
  row0 = __builtin_amdgcn_readfirstlane(a.offsets[e] + at * TM);
  rows = __builtin_amdgcn_readfirstlane(min(min(a.offsets[e + 1], a.out_rows) - row0, TM));
  return true;
}

// Block -> (row tile, feature tile) with NT feature tiles a row tile.  Workgroups go round-robin
// over the 8 XCDs; the feature tiles of one row tile stay on `xcds` of them, so their shared token
// rows are fetched by that many L2s.
__device__ __forceinline__ bool tile_of(const QArgs& a, int NT, int& mt, int& nt) {
  const int ntx = (NT + a.xcds - 1) / a.xcds, groups = 8 / a.xcds;
  const int slot = blockIdx.x >> 3, xcd = blockIdx.x & 7;
  nt = slot % ntx * a.xcds + xcd % a.xcds;
  mt = slot / ntx * groups + xcd / a.xcds;
  return nt < NT;
}
int64_t tile_grid(int64_t tiles, int64_t NT, int xcds) {
  return 8 * ((NT + xcds - 1) / xcds) * ((tiles + 8 / xcds - 1) / (8 / xcds));
}

constexpr uint32_t kOut = 0x80000000u;  // past every range, whatever offset is added to it

// A wave's weights: FT tiles of 16 rows of expert e from output feature f0 on (gated: FT / 2 gate
// tiles, then the up tiles of the same features).
template <int FT, int GROUP, bool GATED>
struct Weights {
  static constexpr int FO = GATED ? FT / 2 : FT, S = 128 / GROUP;
  static_assert(!GATED || FT % 2 == 0, "gate and up tiles in pairs");
  __amdgpu_buffer_rsrc_t cr, sr;
  uint32_t cstep, sstep;  // bytes from a column block to the next
  uint32_t co[FT], so[FT];
  int KC;
  __device__ __forceinline__ Weights(const QArgs& a, int e, int f0, int n, int kg) {
    const int wrows = GATED ? 2 * a.N : a.N;
    KC = (a.K + 127) / 128;
    cstep = wrows * 64;
    sstep = wrows * S * 2;
    cr = buffer_rsrc(a.codes + (int64_t)e * KC * wrows * 4, KC * cstep);
    sr = buffer_rsrc(a.scales + (int64_t)e * KC * wrows * S, KC * sstep);
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      uint32_t r = f0 + f % FO * 16 + n;
      const bool in = (int)r < a.N;
      if (GATED && f >= FO) r += a.N;
      co[f] = in ? (r / 8 * 32 + kg * 8 + r % 8) * 16 : kOut;
      so[f] = in ? r * S * 2 : kOut;
    }
  }
  // column block kc; past the last: zeros, without traffic
  __device__ __forceinline__ void load(int kc, uint4 (&cw)[FT], Scales<GROUP> (&sc)[FT]) const {
    const bool in = kc < KC;
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      cw[f] = buffer_load16(cr, in ? co[f] + kc * cstep : kOut);
      sc[f].load(sr, in ? so[f] + kc * sstep : kOut);
    }
  }
};

// The token rows of a tile: gathered through row_token, or rows row0 .. of A.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t token_rsrc(const QArgs& a, int row0, int rows) {
  return a.row_token ? buffer_rsrc(a.A, (uint32_t)(a.a_rows * a.K * 2))
                     : buffer_rsrc(a.A + (int64_t)row0 * a.K, (uint32_t)rows * a.K * 2);
}
__device__ __forceinline__ uint32_t token_offset(const QArgs& a, int row0, int rows, int r) {
  if (r >= rows) return kOut;
  const int t = a.row_token ? a.row_token[row0 + r] : r;
  return t >= 0 ? (uint32_t)t * a.K * 2 : kOut;
}

// Bias, activation, bf16 and store of a wave's results: rows r0 + 16 rt + 4 kg + j of the tile.
template <int RT, int FT, int ACT>
__device__ __forceinline__ void store_tile(const QArgs& a, const f32x4_t (&acc)[RT][FT], int e,
                                           int row0, int rows, int r0, int f0, int n, int kg) {
  constexpr bool GATED = ACT == kQGated;
  constexpr int FO = GATED ? FT / 2 : FT;
#pragma unroll
  for (int f = 0; f < FO; ++f) {
    const int feat = f0 + f * 16 + n;
    if (feat >= a.N) continue;
    const float b = !GATED && a.bias ? bf16_to_f32(a.bias[(int64_t)e * a.N + feat]) : 0.0f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + rt * 16 + kg * 4 + j;
        float v = acc[rt][f][j];
        if constexpr (GATED)
          v = silu(v) * acc[rt][FO + f][j];
        else
          v = ACT == kQSilu ? silu(v + b) : v + b;
        if (r < rows) a.out[(int64_t)(row0 + r) * a.N + feat] = (bf16_t)pack_bf16x2(v, 0.0f);
      }
  }
}

// ---------------------------------------------------------------- few rows an expert
// A block takes 16 RT token rows of one expert and 16 FT WF of its weight rows; WF waves stand side
// by side on the features, WK share the column blocks (step s: blocks WK s .. WK s + WK - 1), and
// their sums are added in LDS, in wave order.  Weights go from HBM to registers, D steps in
// flight.  STAGED: a step's token rows are loaded into registers two steps ahead and into one of
// two LDS buffers one step ahead, one barrier a step; otherwise (one or two tokens, where the
// barriers cost more than the loads) every wave loads its own.
//
// Bound: the weight stream.  E 8, d 2048, f 8192, 64 tokens, group 32 (75 MB a product): 17.9 us
// up, 23.4 us down, 4.2 and 3.2 TB/s; loading the same codes without products or token rows: 16.8
// and 18.3 us, and 2.3 us of it are an empty launch.  Column blocks outermost in the storage (runs of
// 8 KiB a block of waves) instead of rows outermost: 24.2 -> 20.0 us up, 26.3 -> 22.2 us down.
template <int RT, int FT, int WF, int WK, int D, bool STAGED, int GROUP, int ACT>
__global__ __launch_bounds__(64 * WF * WK) void k_quant_rows(QArgs a) {
  constexpr int S = 128 / GROUP, J = GROUP / 32, W = WF * WK, XL = STAGED ? RT * 4 / WF : RT;
  constexpr bool GATED = ACT == kQGated;
  constexpr int FO = GATED ? FT / 2 : FT;  // output tiles of a wave
  static_assert(!STAGED || RT * 4 % WF == 0, "whole fragments a wave");
  extern __shared__ uint4 smem[];
  auto xs = reinterpret_cast<uint4(*)[WK][RT * 4][64]>(smem);          // [2]
  auto red = reinterpret_cast<f32x4_t(*)[WF][RT * FT][64]>(smem);      // [WK - 1]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wf = wave % WF, wk = wave / WF;
  const int n = lane & 15, kg = lane >> 4;
  int mt, nt, e, row0, rows;
  if (!tile_of(a, (a.N + 16 * FO * WF - 1) / (16 * FO * WF), mt, nt)) return;  // block-uniform
  if (!row_tile<16 * RT>(a, mt, e, row0, rows)) return;                         // block-uniform
  const int f0 = (nt * WF + wf) * FO * 16;
  const Weights<FT, GROUP, GATED> w(a, e, f0, n, kg);
  const int KC = w.KC, steps = (KC + WK - 1) / WK;
  const __amdgpu_buffer_rsrc_t xr = token_rsrc(a, row0, rows);
  // STAGED: fragment i W + wave of a step (its column block, row group and 32 columns); else row
  // group i
  uint32_t xo[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i)
    xo[i] = token_offset(a, row0, rows, (STAGED ? (i * W + wave) / 4 % RT : i) * 16 + n);
  uint4 cw[D][FT], xw[STAGED ? 1 : D][STAGED ? XL : RT * 4];
  Scales<GROUP> sc[D][FT];
  auto load_own = [&](int p, int s) {  // not STAGED: the wave's own column block
#pragma unroll
    for (int i = 0; i < RT * 4; ++i) {
      const int k = (s * WK + wk) * 128 + i % 4 * 32 + kg * 8;
      xw[STAGED ? 0 : p][STAGED ? 0 : i] = buffer_load16(xr, k < a.K ? xo[STAGED ? 0 : i / 4] + k * 2 : kOut);
    }
  };
  auto load_step = [&](int s) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int id = i * W + wave;
      const int k = (s * WK + id / (RT * 4)) * 128 + id % 4 * 32 + kg * 8;
      xw[0][i] = buffer_load16(xr, k < a.K ? xo[i] + k * 2 : kOut);
    }
  };
  auto store_step = [&](int s) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int id = i * W + wave;
      xs[s & 1][id / (RT * 4)][id % (RT * 4)][lane] = xw[0][i];
    }
  };
  f32x4_t acc[RT][FT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int f = 0; f < FT; ++f) acc[rt][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](int p, int s) {
    if (s * WK + wk >= KC) return;  // wave-uniform
#pragma unroll
    for (int g = 0; g < S; ++g) {
      bf16x8_t A[J][RT];
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          A[j][rt] = qfrag(STAGED ? xs[s & 1][wk][rt * 4 + g * J + j][lane]
                                  : xw[STAGED ? 0 : p][STAGED ? 0 : rt * 4 + g * J + j]);
#pragma unroll
      for (int f = 0; f < FT; ++f) {
        const uint32_t c[4] = {cw[p][f].x, cw[p][f].y, cw[p][f].z, cw[p][f].w};
        const float sv = sc[p][f].get(g);
        f32x4_t t[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) t[rt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bf16x8_t B = values_of(c[g * J + j]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            t[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[j][rt], B, t[rt], 0, 0, 0);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][f][i] = fmaf(sv, t[rt][i], acc[rt][f][i]);
        // one tile's conversions at a time: hoisted together they take twice the registers
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  if constexpr (STAGED) load_step(0);
#pragma unroll
  for (int p = 0; p < D - 1; ++p) {
    w.load(p * WK + wk, cw[p], sc[p]);
    if constexpr (!STAGED) load_own(p, p);
  }
  if constexpr (STAGED) {
    store_step(0);
    load_step(1);
    __syncthreads();
  }
  for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
    for (int p = 0; p < D; ++p) {
      const int s = s0 + p;
      if (s >= steps) break;
      w.load((s + D - 1) * WK + wk, cw[(p + D - 1) % D], sc[(p + D - 1) % D]);
      if constexpr (!STAGED) load_own((p + D - 1) % D, s + D - 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(p, s);
      if constexpr (STAGED) {
        store_step(s + 1);
        load_step(s + 2);
        __syncthreads();
      }
    }
  }
  if constexpr (WK > 1) {
    if (wk > 0) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int f = 0; f < FT; ++f) red[wk - 1][wf][rt * FT + f][lane] = acc[rt][f];
    }
    __syncthreads();
    if (wk > 0) return;
    for (int i = 0; i < WK - 1; ++i)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int f = 0; f < FT; ++f) acc[rt][f] += red[i][wf][rt * FT + f][lane];
  }
  store_tile<RT, FT, ACT>(a, acc, e, row0, rows, 0, f0, n, kg);
}

// ---------------------------------------------------------------- many rows an expert
// A block takes 16 RT token rows and 16 FT WF weight rows, a wave 16 FT of them and all token rows:
// each weight is converted once for 16 RT rows.  The fragments of the next (row group, scale
// group) are read from LDS, and the sums of the last one scaled, between the matrix instructions
// of the present one; the scheduling barriers keep the compiler from gathering either at one end
// (gathered: 1.22 ms instead of 0.62 ms on the layer below).
//
// Bound: the matrix instructions and their interleaved conversions and scale products (4 fp32
// products for every CG / 32 matrix instructions), then the latency of the token rows.  E 8, d 2048,
// f 8192, 4096 tokens, top-2: group 128 306 us up and 284 us down, 898 and 968 TFLOP/s (on a
// slower card 317 and 297); group 32 337 and 329 us.  The loads without the products: about 170 us.
template <int WF, int RT, int FT, int GROUP, int ACT>
__global__ __launch_bounds__(64 * WF) void k_quant_tiles(QArgs a) {
  constexpr bool GATED = ACT == kQGated;
  // columns whose sum is scaled at once: groups of 128 in halves, as chains of four dependent matrix
  // instructions leave gaps (group 128 in one: 385 / 344 us, in halves as group 64)
  constexpr int CG = GROUP == 128 ? 64 : GROUP;
  constexpr int FO = GATED ? FT / 2 : FT, S = 128 / CG, J = CG / 32;
  constexpr int XL = RT * 4 / WF, NI = RT * S;  // NI items of a column block: (row group, columns)
  static_assert(RT * 4 % WF == 0, "whole fragments a wave");
  __shared__ uint4 xs[2][RT * 4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  int mt, nt, e, row0, rows;
  if (!tile_of(a, (a.N + 16 * FO * WF - 1) / (16 * FO * WF), mt, nt)) return;  // block-uniform
  if (!row_tile<16 * RT>(a, mt, e, row0, rows)) return;                         // block-uniform
  const int f0 = (nt * WF + wave) * FO * 16;
  const Weights<FT, GROUP, GATED> w(a, e, f0, n, kg);
  const __amdgpu_buffer_rsrc_t xr = token_rsrc(a, row0, rows);
  uint32_t xo[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) xo[i] = token_offset(a, row0, rows, (i * WF + wave) / 4 * 16 + n);
  uint4 cw[FT], xw[XL];
  Scales<GROUP> sc[FT];
  auto load_x = [&](int kc) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int k = kc * 128 + (i * WF + wave) % 4 * 32 + kg * 8;
      xw[i] = buffer_load16(xr, k < a.K ? xo[i] + k * 2 : kOut);
    }
  };
  auto store_x = [&](int kc) {
#pragma unroll
    for (int i = 0; i < XL; ++i) xs[kc & 1][i * WF + wave][lane] = xw[i];
  };
  f32x4_t acc[RT][FT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int f = 0; f < FT; ++f) acc[rt][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  load_x(0);
  w.load(0, cw, sc);
  store_x(0);
  load_x(1);
  __syncthreads();
  for (int kc = 0; kc < w.KC; ++kc) {
    bf16x8_t B[FT][4];
    float s[FT][S];
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      B[f][0] = values_of(cw[f].x);
      B[f][1] = values_of(cw[f].y);
      B[f][2] = values_of(cw[f].z);
      B[f][3] = values_of(cw[f].w);
#pragma unroll
      for (int g = 0; g < S; ++g) s[f][g] = sc[f].get(g * CG / GROUP);
    }
    w.load(kc + 1, cw, sc);
    bf16x8_t A[2][J];
    f32x4_t t[2][FT];
    auto frags = [&](int i) {
#pragma unroll
      for (int j = 0; j < J; ++j) A[i & 1][j] = qfrag(xs[kc & 1][i / S * 4 + i % S * J + j][lane]);
    };
    auto scale = [&](int i) {
#pragma unroll
      for (int f = 0; f < FT; ++f)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          acc[i / S][f][u] = fmaf(s[f][i % S], t[i & 1][f][u], acc[i / S][f][u]);
    };
    frags(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (i + 1 < NI) frags(i + 1);
#pragma unroll
      for (int f = 0; f < FT; ++f) t[i & 1][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int f = 0; f < FT; ++f)
          t[i & 1][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[i & 1][j], B[f][i % S * J + j],
                                                                t[i & 1][f], 0, 0, 0);
      if (i > 0) scale(i - 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    scale(NI - 1);
    store_x(kc + 1);
    load_x(kc + 2);
    __syncthreads();
  }
  store_tile<RT, FT, ACT>(a, acc, e, row0, rows, 0, f0, n, kg);
}

// ---------------------------------------------------------------- choice of the kernel
template <int RT, int FT, int WF, int WK, int D, bool STAGED, int GROUP, int ACT>
hipError_t run_rows(const QArgs& a, int64_t tiles, int64_t NT, hipStream_t st) {
  constexpr size_t x = STAGED ? (size_t)2 * WK * RT * 4096 : 0;
  constexpr size_t r = (size_t)(WK - 1) * WF * RT * FT * 1024;
  constexpr size_t lds = x > r ? x : r;
  static_assert(lds <= 64 * 1024, "LDS without an attribute");
  return launch_timed(k_quant_rows<RT, FT, WF, WK, D, STAGED, GROUP, ACT>,
                      dim3((unsigned)tile_grid(tiles, NT, a.xcds)), dim3(64 * WF * WK), lds, st, a);
}

// Rows an expert on average, and blocks a variant would launch, decide.  Kernel times in us, "up + down"
// or of the product named, random routing, the weights of several layers in turn (more than the
// caches hold):
//  - more than 48 rows: 64 x 256 tiles of 8 waves, once they are one a CU (8 experts, d 2048, f 8192,
//    1024 rows each, group 128: 317 + 295 against 372 + 312 for 32 x 256; 64 experts, d 2048, f 1408,
//    72 rows each: 60 + 52 against 63 + 54; 38 rows each: 41 + 40 against 41 + 38.  At the limit it
//    depends on the blocks: 48 rows each 42 + 41 against 48 + 45 with 384 and 512 tiles, 38 + 33
//    against 31 + 28 for 32 experts of f 2048 with 256); gated, which has no 32 x 128, from 160
//    blocks on (2 experts, d 2048, f 4096, 200 rows each, up: 23.6 against 28.9 for K shared);
//  - at most 6 rows and 512 blocks: 16 token rows by 128 weight rows, waves of twice the width (64
//    experts, d 2048, f 1408, 6 rows each: 22.5 + 20.9 against 23.0 + 22.3 for the 32 x 128; 16 experts of
//    4 rows, d 2048, f 4096, 512 blocks up: 18.9 against 19.1).  Gated by 256, from 256 blocks on (64
//    experts of 4 rows, d 1024, f 1408: 21.5 against 23.5 for 32 x 256 and for 16 x 128 with K shared;
//    128 experts of 6 rows, d 2048, f 768, group 128: 39.3 against 45.3 and 41.0; but 64 experts of 6
//    rows, d 2048, f 1408: 43.5 against 44.8 and 39.3);
//  - else 32 rows x 256 weight rows, from 320 blocks on, 640 for more than 48 rows (2 experts, d 624,
//    f 7400, 2200 rows each, 400 down: 155 against 93 for the next; 8 experts, d 2048, f 8192, 16
//    rows each, 256 up: 21.9 against 20.3; 64 experts, d 2048, f 1408, 24 rows each, 384 up: 29.4
//    against 33.2); gated from 160 on (8 experts, f 4096, 16 rows each, 256 up: 18.1 against 18.7 for
//    the last but one);
//  - else 32 x 128, from 256 blocks on (8 experts, f 8192, 16 rows each, up: 20.3 against 32.4);
//  - else K is shared by groups of waves, 64 weight rows a block.  Four groups for long K: 32 token
//    rows if the blocks, of 16 waves, are one a CU (d 2048, f 8192, 16 rows each, down: 22.0 against
//    27.7 with 16 token rows; 20 rows each, where some CUs get two once an expert has more than 32:
//    60.5 against 54.6 for both products).  Two groups for K below 4096 (8 gated experts, d 2048,
//    f 768, 9 rows each, up: 8.8 against 9.3 with four), of 16 token rows up to 24 rows an expert (24
//    rows each, up: 9.6 against 10.8 with 32 token rows; 64 rows each: 13.1 against 11.9);
//  - few tokens with few such blocks: 16 weight rows a block, K shared by 8 waves that load their own
//    token rows (1 token, f 8192, down: 6.5 against 12.5; 2 rows each, f 1408: 8.8 + 8.5 against
//    7.9 + 5.4, from 128 blocks on therefore not).
// A gated tile holds a gate and an up row per feature: half the features a block.
template <int GROUP, int ACT>
hipError_t run_quant(QArgs a, int64_t rows_ub, hipStream_t st) {
  constexpr bool GATED = ACT == kQGated;
  constexpr int F1 = GATED ? 2 : 1;  // the narrowest wave: one feature tile, or a gate and an up tile
  const int64_t active = rows_ub < a.E ? rows_ub : a.E, mean = (rows_ub + a.E - 1) / a.E;
  auto NT = [&](int wrows) {  // feature tiles of blocks of that many weight rows
    const int64_t f = GATED ? wrows / 2 : wrows;
    return (a.N + f - 1) / f;
  };
  auto likely = [&](int TM) {  // row tiles: a whole and half a tile an expert
    const int64_t t = rows_ub / TM + active / 2;
    return t > active ? t : active;
  };
  auto most = [&](int TM) {  // row tiles, at most
    const int64_t t = rows_ub / TM + a.E;
    return t < rows_ub ? t : rows_ub;
  };
  // few row tiles go over all XCDs; more are dealt to pairs of them
  a.xcds = active < 8 ? 8 : 2;
  if (mean > 48 && NT(256) * likely(64) >= (GATED ? 160 : 256))
    return launch_timed(k_quant_tiles<8, 4, 2, GROUP, ACT>,
                        dim3((unsigned)tile_grid(most(64), NT(256), a.xcds)), dim3(512), 0, st, a);
  if (mean <= 6 && NT(128 * F1) * likely(16) >= 512 / F1)
    return run_rows<1, 2 * F1, 4, 1, GATED ? 2 : 4, true, GROUP, ACT>(a, most(16), NT(128 * F1), st);
  if (NT(256) * likely(32) >= (GATED ? 160 : mean > 48 ? 640 : 320))
    return run_rows<2, 2, 8, 1, 3, true, GROUP, ACT>(a, most(32), NT(256), st);
  if constexpr (!GATED)
    if (NT(128) * likely(32) >= 256)
      return run_rows<2, 1, 8, 1, 2, true, GROUP, ACT>(a, most(32), NT(128), st);
  const bool long_k = a.K >= 4096;
  if (long_k && mean > 8 && NT(64 * F1) * likely(32) <= 256)
    return run_rows<2, F1, 4, 4, 2, true, GROUP, ACT>(a, most(32), NT(64 * F1), st);
  if (mean > 24) return run_rows<2, F1, 4, 2, 2, true, GROUP, ACT>(a, most(32), NT(64 * F1), st);
  if (mean > 8 || NT(64 * F1) * likely(16) >= (mean > 1 ? 128 : 192)) {
    if (long_k) return run_rows<1, F1, 4, 4, 2, true, GROUP, ACT>(a, most(16), NT(64 * F1), st);
    return run_rows<1, F1, 4, 2, 2, true, GROUP, ACT>(a, most(16), NT(64 * F1), st);
  }
  return run_rows<1, F1, 1, 8, 2, false, GROUP, ACT>(a, most(16), NT(16 * F1), st);
}

template <int ACT>
hipError_t run_quant(int group, const QArgs& a, int64_t rows_ub, hipStream_t st) {
  if (rows_ub <= 0) return hipSuccess;
  if (group == 32) return run_quant<32, ACT>(a, rows_ub, st);
  if (group == 64) return run_quant<64, ACT>(a, rows_ub, st);
  return run_quant<128, ACT>(a, rows_ub, st);
}

}  // namespace

hipError_t launch_quant_up(const moe_shape& s, const moe_quantized_experts& q, const void* x,
                           const int32_t* row_token, const int32_t* offsets, void* h,
                           int64_t rows_ub, hipStream_t st) {
  QArgs a = {};
  a.A = (const bf16_t*)x;
  a.row_token = row_token;
  a.offsets = offsets;
  a.codes = (const uint4*)q.w1_codes;
  a.scales = (const bf16_t*)q.w1_scales;
  a.bias = (const bf16_t*)q.b1;
  a.out = (bf16_t*)h;
  a.E = s.n_experts;
  a.N = s.d_ff;
  a.K = s.d_model;
  a.a_rows = s.T;
  a.out_rows = (int)rows_ub;
  return q.gated ? run_quant<kQGated>(q.group, a, rows_ub, st)
                 : run_quant<kQSilu>(q.group, a, rows_ub, st);
}

hipError_t launch_quant_down(const moe_shape& s, const moe_quantized_experts& q, const void* h,
                             const int32_t* offsets, void* y, int64_t rows_ub, hipStream_t st) {
  QArgs a = {};
  a.A = (const bf16_t*)h;
  a.offsets = offsets;
  a.codes = (const uint4*)q.w2_codes;
  a.scales = (const bf16_t*)q.w2_scales;
  a.bias = (const bf16_t*)q.b2;
  a.out = (bf16_t*)y;
  a.E = s.n_experts;
  a.N = s.d_model;
  a.K = s.d_ff;
  a.a_rows = rows_ub;
  a.out_rows = (int)rows_ub;
  return run_quant<kQNone>(q.group, a, rows_ub, st);
}

}  // namespace moe
