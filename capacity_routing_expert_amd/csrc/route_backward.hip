// Backward pass of the router: from the gradients on the top-k gates and on the logits to those
// on the token rows, the router weights and the router bias.
//
//   dp_te = sum of dgates[t, c] over the choices c with ids[t, c] = e
//   dl_te = p_te (dp_te - sum_j p_tj dp_tj) + dlogits_te      p = softmax of the logits
//   dx = dx_add + dl W_r,   dW_r = dl^T x,   db = sum_t dl_t
//
// Bound: HBM, for the expert counts that the library takes in bf16 (x is read once for dW_r, dx
// is written once; 4 T E d flops): T 32768, d 4096, E 8 7.4 us for dl, 104 us for dx (537 MB with
// dx_add and dx), 71 us for dW_r (268 MB), 5.7 us for the sums over the token ranges; T 16384, d 2048,
// E 64 7.9, 33.5, 24.1 and 4.9 us.  dl itself is E values a token, so it goes through memory
// between the kernels: k_route_dlogits writes it once in the two layouts that the matrix
// instructions want (experts contiguous for dx, tokens contiguous for dW_r).
//
// bf16: x and W_r are bf16 as they stand, dl is fp32, and splitting dl into bf16 terms
// (dl = hi + mid + lo, 24 bits) lets v_mfma_f32_16x16x32_bf16 form exact products with fp32
// sums.  dW_r (an fp32 result) takes all three terms; dx, which is rounded to bf16 (2^-8), takes
// two (2^-16 of each dl).  f32: v_mfma_f32_16x16x4f32 on the fp32 values.
#include "router_rows.h"

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8_t frag(uint4 v) { return __builtin_bit_cast(bf16x8_t, v); }

constexpr int kTT = 64;           // tokens of a k_route_dlogits tile
constexpr int kMaxDlBlocks = 256; // blocks of k_route_dlogits (partials of db)
constexpr int kCols = 128;        // columns of a wave in the bf16 kernels: 16 lanes x 8
constexpr int kColsF32 = 64;      // ... and in the f32 ones: 4 tiles of 16

// Workspace of the backward pass; each part on a 256-byte boundary.
struct BackwardLayout {
  int64_t Tp;        // tokens rounded up to whole tiles
  int64_t EK;        // experts of a row of dl_x, rounded up (bf16: 8, f32: 4)
  size_t dl_x;       // bf16: [2 terms][Tp][EK] bf16; f32: [Tp][EK] fp32
  size_t dl_w;       // bf16: [3 terms][E][Tp] bf16; f32: [E][Tp] fp32
  size_t valid;      // [Tp] u8: 1 for a valid token
  size_t db_part;    // [dl_blocks][E] fp32
  size_t dw_part;    // [splits][E][d] fp32
  int64_t dl_blocks;
  int64_t splits;    // token ranges of dW_r
  size_t total;
};

BackwardLayout backward_layout(const moe_shape& s) {
  BackwardLayout L;
  const bool bf = s.dtype == MOE_BF16;
  const int64_t E = s.n_experts, d = s.d_model;
  L.Tp = (s.T + kTT - 1) / kTT * kTT;
  L.EK = bf ? (E + 7) / 8 * 8 : (E + 3) / 4 * 4;
  const int64_t tiles = L.Tp / kTT;
  L.dl_blocks = tiles < kMaxDlBlocks ? tiles : kMaxDlBlocks;
  // blocks of dW_r: column tiles x groups of 64 experts x token ranges, and at least 128 tokens a
  // range.  bf16: about one a compute unit (T 16384, E 64, d 2048: 25 us, with twice the blocks 33,
  // as each writes a partial dW_r of its own); f32, whose waves have half the bytes on their
  // way: three (the whole pass at T 8192, E 128, d 4096: 285 us, with two 343, with one 507)
  const int64_t cols = bf ? kCols : kColsF32;
  const int64_t base = (d + cols - 1) / cols * ((E + 63) / 64);
  int64_t splits = ((bf ? 256 : 768) + base - 1) / base;
  const int64_t most = (s.T + 127) / 128;
  if (splits > most) splits = most;
  L.splits = splits < 1 ? 1 : splits;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at_ = o;
    o = (o + bytes + 255) & ~(size_t)255;
    return at_;
  };
  L.dl_x = take((size_t)L.Tp * L.EK * 4);
  L.dl_w = take((size_t)L.Tp * E * (bf ? 6 : 4));
  L.valid = take((size_t)L.Tp);
  L.db_part = take((size_t)L.dl_blocks * E * 4);
  L.dw_part = take((size_t)L.splits * E * d * 4);
  L.total = o;
  return L;
}

// ---------------------------------------------------------------- dl
struct DlArgs {
  const float* logits;
  const int32_t* ids;
  const float* dgates;   // or NULL
  const float* dlogits;  // or NULL
  const uint8_t* mask;   // or NULL
  int64_t T, Tp;
  int E, EK, k;
  void* dl_x;      // or NULL
  void* dl_w;      // or NULL
  uint8_t* valid;  // or NULL
  float* db_part;  // or NULL
};

// Block -> (column tile, token range) with `cols` column tiles a range.  Workgroups go round-robin
// over the 8 XCDs; the column tiles of one range stay on one XCD, so dl, which all of them read,
// comes through one L2.
__device__ __forceinline__ bool range_of(int cols, int64_t ranges, int& col, int64_t& range) {
  const int slot = blockIdx.x >> 3, xcd = blockIdx.x & 7;
  col = slot % cols;
  range = (int64_t)(slot / cols) * 8 + xcd;
  return range < ranges;
}
int64_t range_grid(int64_t cols, int64_t ranges) { return 8 * cols * ((ranges + 7) / 8); }

constexpr int kDlThreads = 512;
constexpr int kDlChoices = 8;  // choices staged at a time

// One block takes tiles of 64 tokens: softmax gradients of the tile's rows into LDS, [expert]
// [token] with a pitch of 65 words, then both layouts from there.  Rows past T and masked rows
// are zero, so the product kernels need no guards on dl.  Latency-bound: 64 tokens a block are
// few loads, so the logits of the first rows and the choices are asked for before anything waits.
template <typename Row, bool BF>
__global__ __launch_bounds__(kDlThreads) void k_route_dlogits(DlArgs a) {
  constexpr int LPT = Row::LPT, NV = Row::NV, TPW = Row::TPW, P = kTT + 1, NW = kDlThreads / 64;
  extern __shared__ float tile[];  // [E][P], then [E][8] partial sums of db
  __shared__ int sid[kTT * kDlChoices];
  __shared__ float sgate[kTT * kDlChoices];
  const int E = a.E, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane % LPT;
  float* dbs = tile + E * P;
  float db = 0.0f;
  for (int64_t tb = (int64_t)blockIdx.x * kTT; tb < a.Tp; tb += (int64_t)gridDim.x * kTT) {
    float p[NV], in[NV];
    bool valid = false;
    auto load = [&](int g) {  // rows g .. g + TPW - 1 of the tile
      const int tl = g + lane / LPT;
      const int64_t t = tb + tl;
      valid = tl < kTT && t < a.T && (!a.mask || a.mask[t]);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        p[i] = -INFINITY;  // not valid: probabilities 0
        in[i] = 0.0f;
      }
      if (valid && a.dgates) Row::load(a.logits + t * E, E, l, -INFINITY, p);
      if (valid && a.dlogits) Row::load(a.dlogits + t * E, E, l, 0.0f, in);
    };
    load(wave * TPW);
    // gate gradients scattered to their experts: one thread a token, choices in order
    if (a.dgates) {
      for (int i = tid; i < E * P; i += kDlThreads) tile[i] = 0.0f;
      for (int c0 = 0; c0 < a.k; c0 += kDlChoices) {
        const int tl = tid / kDlChoices, c = c0 + tid % kDlChoices;
        const int64_t t = tb + tl;
        int id = -1;
        float gate = 0.0f;
        if (c < a.k && t < a.T && (!a.mask || a.mask[t])) {
          id = a.ids[t * a.k + c];
          gate = a.dgates[t * a.k + c];
        }
        sid[tid] = id;
        sgate[tid] = gate;
        __syncthreads();
        if (tid < kTT) {
#pragma unroll
          for (int j = 0; j < kDlChoices; ++j) {
            const int e = sid[tid * kDlChoices + j];
            if ((unsigned)e < (unsigned)E) tile[e * P + tid] += sgate[tid * kDlChoices + j];
          }
        }
        __syncthreads();
      }
    }
    for (int g = wave * TPW; g < kTT; g += NW * TPW) {
      const int tl = g + lane / LPT;
      float dl[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) dl[i] = 0.0f;
      if (a.dgates) {
        float dot = 0.0f;
        Row::softmax(p);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = Row::expert(l, i);
          dl[i] = tl < kTT && e < E ? tile[e * P + tl] : 0.0f;
          dot += p[i] * dl[i];
        }
        dot = row_sum<LPT>(dot);
#pragma unroll
        for (int i = 0; i < NV; ++i) dl[i] = p[i] * (dl[i] - dot);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) dl[i] = valid ? dl[i] + in[i] : 0.0f;
      if (tl < kTT) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = Row::expert(l, i);
          if (e < E) tile[e * P + tl] = dl[i];
        }
        if (l == 0 && a.valid) a.valid[tb + tl] = valid;
      }
      load(g + NW * TPW);
    }
    __syncthreads();
    if (a.dl_x) {
      constexpr int W = BF ? 8 : 4;  // experts of a 16-byte chunk
      const int chunks = a.EK / W;
      for (int i = tid; i < kTT * chunks; i += kDlThreads) {
        const int tl = i / chunks, e0 = i % chunks * W;
        float v[W];
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = e0 + j < E ? tile[(e0 + j) * P + tl] : 0.0f;
        const int64_t at = (tb + tl) * a.EK + e0;
        if constexpr (BF) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            hi[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
            lo[j] = pack_bf16x2(v[2 * j] - __uint_as_float(hi[j] << 16),
                                v[2 * j + 1] - __uint_as_float(hi[j] & 0xFFFF0000u));
          }
          bf16_t* o = static_cast<bf16_t*>(a.dl_x);
          *reinterpret_cast<uint4*>(o + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(o + a.Tp * a.EK + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(a.dl_x) + at) =
              make_float4(v[0], v[1], v[2], v[3]);
        }
      }
    }
    if (a.dl_w || a.db_part) {
      for (int i = tid; i < E * (kTT / 8); i += kDlThreads) {
        const int e = i / (kTT / 8), t0 = i % (kTT / 8) * 8;
        float v[8], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = tile[e * P + t0 + j];
          sum += v[j];
        }
        if (a.db_part) dbs[i] = sum;
        if (!a.dl_w) continue;
        const int64_t at = (int64_t)e * a.Tp + tb + t0;
        if constexpr (BF) {
          bf16_t* o = static_cast<bf16_t*>(a.dl_w);
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
              v[2 * j] -= __uint_as_float(w[j] << 16);
              v[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
            }
            *reinterpret_cast<uint4*>(o + term * (int64_t)E * a.Tp + at) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float* o = static_cast<float*>(a.dl_w) + at;
          *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
    __syncthreads();  // the tile is overwritten by the next one
    if (a.db_part && tid < E)
      for (int j = 0; j < kTT / 8; ++j) db += dbs[tid * (kTT / 8) + j];
  }
  if (a.db_part && tid < E) a.db_part[(int64_t)blockIdx.x * E + tid] = db;
}

// Eight rows of eight bf16 columns, one row a uint4, transposed: out[i] holds column i of the
// rows, row 0 in the lowest half.
__device__ __forceinline__ void transpose8x8(const uint4 (&r)[8], uint4 (&out)[8]) {
  const uint32_t* in[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) in[j] = reinterpret_cast<const uint32_t*>(&r[j]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
      w[m] = __builtin_amdgcn_perm(in[2 * m + 1][i / 2], in[2 * m][i / 2],
                                   i % 2 ? 0x07060302u : 0x05040100u);
    out[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------- dx, bf16
// A wave takes 32 tokens x 128 columns.  Lane n of a 16-lane group owns columns 8 n .. 8 n + 7:
// column 8 n + i belongs to MFMA tile i, so the eight tiles of a lane are one 16-byte store of
// a row.  The block's W_r columns sit in LDS as ready fragments ([32-expert step][tile][lane]),
// and its four waves walk the token tiles of the block's range.
__global__ __launch_bounds__(256) void k_route_dx_bf16(const bf16_t* __restrict__ dl,
                                                       const bf16_t* __restrict__ w,
                                                       const bf16_t* add, bf16_t* dx, int64_t T,
                                                       int64_t Tp, int d, int E, int EK,
                                                       int64_t ranges) {
  extern __shared__ uint4 wfrag[];  // [KS][8][64]
  int cb;
  int64_t range;
  if (!range_of((d + kCols - 1) / kCols, ranges, cb, range)) return;  // block-uniform
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, kg = lane >> 4;
  const int KS = (E + 31) / 32;
  const int col = cb * kCols + 8 * n;
  const bool incol = col < d;
  for (int ks = wave; ks < KS; ks += 4) {
    uint4 r[8], o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = ks * 32 + kg * 8 + j;
      r[j] = make_uint4(0, 0, 0, 0);
      if (e < E && incol) r[j] = *reinterpret_cast<const uint4*>(w + (int64_t)e * d + col);
    }
    transpose8x8(r, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) wfrag[(ks * 8 + i) * 64 + lane] = o[i];
  }
  __syncthreads();
  const int64_t step = ranges * 128;
  // chunks of experts past EK repeat the last one's: they meet zero rows of W_r
  uint4 A[2][2];
  auto load = [&](int64_t t0, int ks) {
    const int64_t tt = min(t0, Tp - 32);
    const int e = min(ks * 32 + kg * 8, EK - 8);
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int term = 0; term < 2; ++term)
        A[rt][term] = *reinterpret_cast<const uint4*>(
            dl + ((int64_t)term * Tp + tt + rt * 16 + n) * EK + e);
  };
  uint4 next[2][4];
  auto load_add = [&](int64_t t0) {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + rt * 16 + kg * 4 + j;
        next[rt][j] = make_uint4(0, 0, 0, 0);
        if (add && t < T && incol) next[rt][j] = *reinterpret_cast<const uint4*>(add + t * d + col);
      }
  };
  int64_t t0 = range * 128 + wave * 32;
  load(t0, 0);
  load_add(t0);
  for (; t0 < T; t0 += step) {
    uint4 ad[2][4];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int j = 0; j < 4; ++j) ad[rt][j] = next[rt][j];
    load_add(t0 + step);
    f32x4_t acc[2][8];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[rt][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int ks = 0; ks < KS; ++ks) {
      bf16x8_t C[2][2];
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int term = 0; term < 2; ++term) C[rt][term] = frag(A[rt][term]);
      const bool last = ks + 1 == KS;
      load(last ? t0 + step : t0, last ? 0 : ks + 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bf16x8_t B = frag(wfrag[(ks * 8 + i) * 64 + lane]);
#pragma unroll
        for (int rt = 0; rt < 2; ++rt)
#pragma unroll
          for (int term = 1; term >= 0; --term)  // the small term first
            acc[rt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(C[rt][term], B, acc[rt][i], 0, 0,
                                                                 0);
      }
    }
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + rt * 16 + kg * 4 + j;
        if (t >= T || !incol) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = acc[rt][i][j];
        if (add) {
          const uint32_t q[4] = {ad[rt][j].x, ad[rt][j].y, ad[rt][j].z, ad[rt][j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] += __uint_as_float(q[i] << 16);
            v[2 * i + 1] += __uint_as_float(q[i] & 0xFFFF0000u);
          }
        }
        *reinterpret_cast<uint4*>(dx + t * d + col) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
      }
  }
}

// ---------------------------------------------------------------- dW_r, bf16
// A wave holds 16 MT experts x 128 columns of dW_r in accumulators and walks 32-token steps of
// its block's range, the next step's loads in flight during the present one's products.  The token
// axis is the contraction, so x enters transposed: a lane loads 8 rows of 8 columns (16-byte
// loads, 256 contiguous bytes a row over 16 lanes) and 32 byte permutations make its eight
// fragments, tile i holding columns 8 n + i.  The four waves take the steps in turn and are added
// in wave order; token ranges are added by k_route_reduce.  valid: NULL when no token is masked.
template <int MT>
__global__ __launch_bounds__(256) void k_route_dw_bf16(const bf16_t* __restrict__ dl,
                                                       const bf16_t* __restrict__ x,
                                                       const uint8_t* __restrict__ valid,
                                                       float* __restrict__ out, int64_t T,
                                                       int64_t Tp, int d, int E, int64_t per,
                                                       int64_t ranges) {
  __shared__ float4 red[2][MT * 8][64];
  int cb;
  int64_t range;
  if (!range_of((d + kCols - 1) / kCols, ranges, cb, range)) return;  // block-uniform
  const int e0 = blockIdx.y * (MT * 16);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  const int col = cb * kCols + 8 * n;
  const bool incol = col < d;
  f32x4_t acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[m][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t ts = range * per, te = ts + per < T ? ts + per : T;
  const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(x, (uint32_t)(T * d * 2));  // below 2 GiB
  const bf16_t* dp[MT];  // rows of experts past E repeat the last one's; they are not stored
#pragma unroll
  for (int m = 0; m < MT; ++m) dp[m] = dl + (int64_t)min(e0 + m * 16 + n, E - 1) * Tp + kg * 8;
  uint4 r[8], A[MT][3];
  // a masked token's row is not read (whatever it holds counts as zeros)
  auto mask_of = [&](int64_t t0) -> uint2 {
    if (valid) return *reinterpret_cast<const uint2*>(valid + min(t0, Tp - 32) + kg * 8);
    return make_uint2(0x01010101u, 0x01010101u);
  };
  auto load = [&](int64_t t0, uint2 ok) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t t = t0 + kg * 8 + j;
      const bool in = incol && t < te && ((j < 4 ? ok.x : ok.y) >> (8 * (j & 3)) & 1);
      r[j] = buffer_load16(xr, in ? (uint32_t)(t * d + col) * 2 : 0x80000000u);
    }
    const int64_t td = min(t0, Tp - 32);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int term = 0; term < 3; ++term)
        A[m][term] = *reinterpret_cast<const uint4*>(dp[m] + (int64_t)term * E * Tp + td);
  };
  int64_t t0 = ts + wave * 32;
  uint2 ok = mask_of(t0);
  load(t0, ok);
  ok = mask_of(t0 + 128);
  for (; t0 < te; t0 += 128) {
    uint4 B[8], C[MT][3];
    transpose8x8(r, B);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int term = 0; term < 3; ++term) C[m][term] = A[m][term];
    load(t0 + 128, ok);
    ok = mask_of(t0 + 256);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int term = 2; term >= 0; --term)  // the small terms first
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(C[m][term]), frag(B[i]),
                                                              acc[m][i], 0, 0, 0);
  }
  // waves 2, 3 into 0, 1, then 1 into 0
  for (int half = 2; half >= 1; half >>= 1) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          red[wave - half][m * 8 + i][lane] =
              make_float4(acc[m][i][0], acc[m][i][1], acc[m][i][2], acc[m][i][3]);
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 o = red[wave][m * 8 + i][lane];
          acc[m][i][0] += o.x;
          acc[m][i][1] += o.y;
          acc[m][i][2] += o.z;
          acc[m][i][3] += o.w;
        }
    }
    __syncthreads();
  }
  if (wave || !incol) return;
  float* o = out + range * E * d;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + m * 16 + kg * 4 + j;
      if (e >= E) continue;
      float4* q = reinterpret_cast<float4*>(o + (int64_t)e * d + col);
      q[0] = make_float4(acc[m][0][j], acc[m][1][j], acc[m][2][j], acc[m][3][j]);
      q[1] = make_float4(acc[m][4][j], acc[m][5][j], acc[m][6][j], acc[m][7][j]);
    }
}

// ---------------------------------------------------------------- fp32
// The sum of a matrix instruction does not mind the order of its terms, so lane group kg takes experts
// (dx) or tokens (dW_r) 4 kg .. 4 kg + 3 of 16, one 16-byte load, and tile i of four holds columns
// 4 n + i: rows of x, W_r and dx move in 16-byte pieces, 256 B a row.  VEC: d is a multiple of 4 and the
// arrays lie on 16 bytes.
// T 1970, d 4024, E 11, with dx_add: dx 13.5 us (95 MB), dW_r 12.8 us (32 MB); with a dword a lane
// and loads behind branches 57 us for the whole pass instead of 32.  T 8192, d 4096, E 128, where the
// matrix instructions (153 TFLOP/s in a large product) need 56 us each: dx 95 us, dW_r 156 us (x read
// once for each 64 experts; 6 token ranges, on 6 of the 8 XCDs).
template <bool VEC>
__device__ __forceinline__ float4 load_cols(const float* row, int c, int d) {
  if constexpr (VEC) return c < d ? *reinterpret_cast<const float4*>(row + c) : make_float4(0, 0, 0, 0);
  return make_float4(c < d ? row[c] : 0.0f, c + 1 < d ? row[c + 1] : 0.0f,
                     c + 2 < d ? row[c + 2] : 0.0f, c + 3 < d ? row[c + 3] : 0.0f);
}
template <bool VEC>
__device__ __forceinline__ void store_cols(float* row, int c, int d, float4 v) {
  if constexpr (VEC) {
    if (c < d) *reinterpret_cast<float4*>(row + c) = v;
  } else {
    if (c < d) row[c] = v.x;
    if (c + 1 < d) row[c + 1] = v.y;
    if (c + 2 < d) row[c + 2] = v.z;
    if (c + 3 < d) row[c + 3] = v.w;
  }
}

// dx: a wave takes 16 tokens x 64 columns at a time; the block's columns of W_r stay in LDS.
template <bool VEC>
__global__ __launch_bounds__(256) void k_route_dx_f32(const float* __restrict__ dl,
                                                      const float* __restrict__ w,
                                                      const float* add, float* dx, int64_t T,
                                                      int d, int E, int EK, int64_t ranges) {
  extern __shared__ float4 wl[];  // [experts, up to whole 16][16]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, kg = lane >> 4;
  int col;
  int64_t range;
  if (!range_of((d + kColsF32 - 1) / kColsF32, ranges, col, range)) return;  // block-uniform
  const int c = col * kColsF32 + n * 4, EG = (E + 15) / 16;
  for (int i = threadIdx.x; i < EG * 256; i += 256)  // i % 16 is this thread's n
    wl[i] = i / 16 < E ? load_cols<VEC>(w + (int64_t)(i / 16) * d, c, d) : make_float4(0, 0, 0, 0);
  __syncthreads();
  for (int64_t t0 = range * 64 + wave * 16; t0 < T; t0 += ranges * 64) {
    const float* row = dl + (t0 + n) * EK;  // rows up to Tp and experts up to EK are there
    float4 in[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + kg * 4 + j;
      in[j] = add && t < T ? load_cols<VEC>(add + t * d, c, d) : make_float4(0, 0, 0, 0);
    }
    f32x4_t acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int g = 0; g < EG; ++g) {
      const int e = g * 16 + kg * 4;
      const float4 a = e < EK ? *reinterpret_cast<const float4*>(row + e) : make_float4(0, 0, 0, 0);
      const float A[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float4 b = wl[(e + s) * 16 + n];
        acc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(A[s], b.x, acc[0], 0, 0, 0);
        acc[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(A[s], b.y, acc[1], 0, 0, 0);
        acc[2] = __builtin_amdgcn_mfma_f32_16x16x4f32(A[s], b.z, acc[2], 0, 0, 0);
        acc[3] = __builtin_amdgcn_mfma_f32_16x16x4f32(A[s], b.w, acc[3], 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + kg * 4 + j;
      if (t < T)
        store_cols<VEC>(dx + t * d, c, d,
                        make_float4(acc[0][j] + in[j].x, acc[1][j] + in[j].y, acc[2][j] + in[j].z,
                                    acc[3][j] + in[j].w));
    }
  }
}

// dW_r: a wave takes 64 experts x 64 columns at most and 16 tokens at a time, the next 16 on their
// way; no load stands behind a branch, as the waits at its end would be for every load before it.
template <int MT, bool VEC>
__global__ __launch_bounds__(256) void k_route_dw_f32(const float* __restrict__ dl,
                                                      const float* __restrict__ x,
                                                      const uint8_t* __restrict__ valid,
                                                      float* __restrict__ out, int64_t T,
                                                      int64_t Tp, int d, int E, int64_t per,
                                                      int64_t ranges) {
  __shared__ float4 red[2][MT * 4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  int col;
  int64_t range;
  if (!range_of((d + kColsF32 - 1) / kColsF32, ranges, col, range)) return;  // block-uniform
  const int c = col * kColsF32 + n * 4, e0 = blockIdx.y * 64;
  f32x4_t acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t ts = range * per, te = ts + per < T ? ts + per : T;
  const float* dp[MT];  // rows of experts past E repeat the last one's; they are not stored
#pragma unroll
  for (int m = 0; m < MT; ++m) dp[m] = dl + (int64_t)min(e0 + m * 16 + n, E - 1) * Tp + kg * 4;
  float4 r[4], A[MT];
  // a masked token's row is not read (whatever it holds counts as zeros)
  auto mask_of = [&](int64_t t0) -> uint32_t {
    return valid ? *reinterpret_cast<const uint32_t*>(valid + min(t0, Tp - 16) + kg * 4) : 0x01010101u;
  };
  auto load = [&](int64_t t0, uint32_t ok) {
    const int rows = t0 < te ? (int)min(te - t0, (int64_t)16) : 0;
    const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(x + (rows ? t0 : 0) * d, (uint32_t)rows * d * 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = kg * 4 + j < rows && (ok >> (8 * j) & 1);
      const uint32_t at = (uint32_t)((kg * 4 + j) * d + c) * 4;
      if constexpr (VEC) {
        const uint4 v = buffer_load16(xr, in && c < d ? at : 0x80000000u);
        r[j] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                           __uint_as_float(v.w));
      } else {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = buffer_load_f32(xr, in && c + i < d ? at + i * 4 : 0x80000000u);
        r[j] = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
    const int64_t td = min(t0, Tp - 16);
#pragma unroll
    for (int m = 0; m < MT; ++m) A[m] = *reinterpret_cast<const float4*>(dp[m] + td);
  };
  int64_t t0 = ts + wave * 16;
  uint32_t ok = mask_of(t0);
  load(t0, ok);
  ok = mask_of(t0 + 64);
  for (; t0 < te; t0 += 64) {
    float4 B[4], C[MT];
#pragma unroll
    for (int j = 0; j < 4; ++j) B[j] = r[j];
#pragma unroll
    for (int m = 0; m < MT; ++m) C[m] = A[m];
    const uint32_t now = ok;
    ok = mask_of(t0 + 128);
    __builtin_amdgcn_sched_barrier(0);
    load(t0 + 64, now);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float a = j == 0 ? C[m].x : j == 1 ? C[m].y : j == 2 ? C[m].z : C[m].w;
        acc[m][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, B[j].x, acc[m][0], 0, 0, 0);
        acc[m][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, B[j].y, acc[m][1], 0, 0, 0);
        acc[m][2] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, B[j].z, acc[m][2], 0, 0, 0);
        acc[m][3] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, B[j].w, acc[m][3], 0, 0, 0);
      }
  }
  for (int half = 2; half >= 1; half >>= 1) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[wave - half][m * 4 + i][lane] =
              make_float4(acc[m][i][0], acc[m][i][1], acc[m][i][2], acc[m][i][3]);
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 o = red[wave][m * 4 + i][lane];
          acc[m][i][0] += o.x;
          acc[m][i][1] += o.y;
          acc[m][i][2] += o.z;
          acc[m][i][3] += o.w;
        }
    }
    __syncthreads();
  }
  if (wave) return;
  float* o = out + range * E * d;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + m * 16 + kg * 4 + j;
      if (e < E)
        store_cols<VEC>(o + (int64_t)e * d, c, d,
                        make_float4(acc[m][0][j], acc[m][1][j], acc[m][2][j], acc[m][3][j]));
    }
}

// ---------------------------------------------------------------- sums of partial results
// out[i] = sum over p of part[p][i], in order of p; blocks past dw_blocks do db.  No parts: zeros.
__global__ __launch_bounds__(256) void k_route_reduce(const float* __restrict__ dw_part,
                                                      int64_t splits, int64_t n,
                                                      float* __restrict__ dw, int dw_blocks,
                                                      const float* __restrict__ db_part,
                                                      int64_t db_parts, int E,
                                                      float* __restrict__ db) {
  if ((int)blockIdx.x < dw_blocks) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)dw_blocks * 256) {
      float s = 0.0f;
#pragma unroll 8
      for (int64_t p = 0; p < splits; ++p) s += dw_part[p * n + i];
      dw[i] = s;
    }
    return;
  }
  // db: 256 / EG threads a column, added in order
  __shared__ float red[256];
  int EG = 1;
  while (EG < E) EG <<= 1;
  const int e = threadIdx.x % EG, r0 = threadIdx.x / EG, rows = 256 / EG;
  float s = 0.0f;
  if (e < E) {
#pragma unroll 16
    for (int64_t p = r0; p < db_parts; p += rows) s += db_part[p * E + e];
  }
  red[threadIdx.x] = s;
  __syncthreads();
  if ((int)threadIdx.x < E) {
    s = 0.0f;
    for (int r = 0; r < rows; ++r) s += red[r * EG + threadIdx.x];
    db[threadIdx.x] = s;
  }
}

}  // namespace

size_t route_backward_ws_bytes(const moe_shape& s) { return backward_layout(s).total; }

hipError_t launch_route_backward(const moe_shape& s, const void* x, const void* w,
                                 const float* logits, const int32_t* ids, const float* dgates,
                                 const float* dlogits, const uint8_t* mask, const void* dx_add,
                                 void* dx, float* dw, float* db, void* ws, hipStream_t st) {
  const BackwardLayout L = backward_layout(s);
  char* b = static_cast<char*>(ws);
  const int E = s.n_experts, d = s.d_model;
  const bool bf = s.dtype == MOE_BF16;
  float* dw_part = L.splits > 1 ? reinterpret_cast<float*>(b + L.dw_part) : dw;
  float* db_part = L.dl_blocks > 1 ? reinterpret_cast<float*>(b + L.db_part) : db;
  hipError_t err;
  if (s.T > 0) {
    DlArgs a = {};
    a.logits = logits;
    a.ids = ids;
    a.dgates = dgates;
    a.dlogits = dlogits;
    a.mask = mask;
    a.T = s.T;
    a.Tp = L.Tp;
    a.E = E;
    a.EK = (int)L.EK;
    a.k = s.top_k;
    a.dl_x = dx ? b + L.dl_x : nullptr;
    a.dl_w = dw ? b + L.dl_w : nullptr;
    a.valid = mask ? reinterpret_cast<uint8_t*>(b + L.valid) : nullptr;
    a.db_part = db ? db_part : nullptr;
    const bool vec = E % 4 == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)dlogits % 16 == 0;
    err = with_router_row(E, vec, [&](auto row) -> hipError_t {
      using Row = decltype(row);
      auto kern = bf ? k_route_dlogits<Row, true> : k_route_dlogits<Row, false>;
      const int lds = E * (kTT + 1 + kTT / 8) * 4;
      if (lds > 60 * 1024) {
        static std::atomic<bool> done_bf[kMaxDevices], done_f32[kMaxDevices];
        if (hipError_t e = allow_dynamic_lds((const void*)kern, 256 * (kTT + 1 + kTT / 8) * 4, bf ? done_bf : done_f32);
            e != hipSuccess)
          return e;
      }
      hipLaunchKernelGGL(kern, dim3((unsigned)L.dl_blocks), dim3(kDlThreads), lds, st, a);
      return hipGetLastError();
    });
    if (err != hipSuccess) return err;
    const int64_t cols = bf ? kCols : kColsF32, ct = (d + cols - 1) / cols;
    const int64_t rows = bf ? 128 : 64;  // tokens of a dx block at a time
    int64_t tb = (s.T + rows - 1) / rows;
    if (tb > (1024 + ct - 1) / ct) tb = (1024 + ct - 1) / ct;
    int64_t per = (s.T + L.splits - 1) / L.splits;
    per = (per + 127) / 128 * 128;
    const uint8_t* valid = mask ? reinterpret_cast<const uint8_t*>(b + L.valid) : nullptr;
    const int e_groups = (E + 63) / 64;
    // one launch for both products was slower: reads alone and reads with writes mixed on the same
    // channels (T 16384, E 64: 71 us against 33 + 25)
    if (bf && dx) {
      hipLaunchKernelGGL(k_route_dx_bf16, dim3((unsigned)range_grid(ct, tb)), dim3(256),
                         (size_t)(E + 31) / 32 * 8192, st, (const bf16_t*)(b + L.dl_x),
                         (const bf16_t*)w, (const bf16_t*)dx_add, (bf16_t*)dx, s.T, L.Tp, d, E,
                         (int)L.EK, tb);
      if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    if (bf && dw) {
      auto run = [&](auto kern, int experts) {  // of a wave
        hipLaunchKernelGGL(kern,
                           dim3((unsigned)range_grid(ct, L.splits),
                                (unsigned)((E + experts - 1) / experts)),
                           dim3(256), 0, st, (const bf16_t*)(b + L.dl_w), (const bf16_t*)x, valid,
                           dw_part, s.T, L.Tp, d, E, per, L.splits);
        return hipGetLastError();
      };
      // short ranges are latency: waves of 32 experts, two a SIMD (whole pass with 64 / 32 experts a
      // wave, d 2048, E 64: T 512 25.5 / 22.4 us, T 4096 35.9 / 34.3, T 16384, 1024 tokens a range,
      // 69.0 / 71.2)
      err = E <= 16                 ? run(k_route_dw_bf16<1>, 16)
            : E <= 32 || per <= 512 ? run(k_route_dw_bf16<2>, 32)
                                    : run(k_route_dw_bf16<4>, 64);
      if (err != hipSuccess) return err;
    }
    if (!bf) {
      auto run = [&](auto vec) {
        constexpr bool VEC = decltype(vec)::value;
        if (dx) {
          hipLaunchKernelGGL(k_route_dx_f32<VEC>, dim3((unsigned)range_grid(ct, tb)), dim3(256),
                             (size_t)(E + 15) / 16 * 4096, st, (const float*)(b + L.dl_x),
                             (const float*)w, (const float*)dx_add, (float*)dx, s.T, d, E,
                             (int)L.EK, tb);
          if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        }
        if (!dw) return hipSuccess;
        auto dw_run = [&](auto kern) {
          hipLaunchKernelGGL(kern, dim3((unsigned)range_grid(ct, L.splits), (unsigned)e_groups),
                             dim3(256), 0, st, (const float*)(b + L.dl_w), (const float*)x, valid,
                             dw_part, s.T, L.Tp, d, E, per, L.splits);
          return hipGetLastError();
        };
        return E <= 16   ? dw_run(k_route_dw_f32<1, VEC>)
               : E <= 32 ? dw_run(k_route_dw_f32<2, VEC>)
                         : dw_run(k_route_dw_f32<4, VEC>);
      };
      // 16-byte pieces where every row starts on one (fp32 arrays need 4 bytes)
      auto at16 = [](const void* p) { return (uintptr_t)p % 16 == 0; };
      const bool vec16 = d % 4 == 0 && at16(x) && at16(w) && at16(dx) && at16(dx_add) && at16(dw);
      err = vec16 ? run(std::true_type()) : run(std::false_type());
      if (err != hipSuccess) return err;
    }
  }
  const bool sum_dw = dw && (L.splits > 1 || s.T == 0);
  const bool sum_db = db && L.dl_blocks != 1;
  if (!sum_dw && !sum_db) return hipSuccess;
  const int64_t n = (int64_t)E * d;
  int64_t blocks = sum_dw ? (n + 255) / 256 : 0;
  if (blocks > 4096) blocks = 4096;
  hipLaunchKernelGGL(k_route_reduce, dim3((unsigned)(blocks + (sum_db ? 1 : 0))), dim3(256), 0, st,
                     dw_part, s.T > 0 ? L.splits : 0, n, dw, (int)blocks, db_part,
                     s.T > 0 ? L.dl_blocks : 0, E, db);
  return hipGetLastError();
}

}  // namespace moe
