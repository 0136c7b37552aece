// Balance loss of the router, per-expert counts and the gradient on the logits.
//
// n valid tokens (token_mask), c_e assignments of valid tokens to expert e, p_t the softmax of
// token t's logits, S_e = sum of p_te over the valid tokens:
//   loss       = coef E sum_e (c_e / (n k)) (S_e / n)
//   dlogits_te = grad_scale coef E / (n k n) p_te (c_e - sum_j p_tj c_j)
// (the counts are constants of the gradient, so the gradient needs the counts but not S, and one
// pass over the logits gives both).  Only differences of counts matter in the gradient, as the
// p_tj sum to 1: counts are taken from the smallest one, which makes equal counts give exact
// zeros and keeps the subtraction's error relative to the differences.
//
// Bound: reading the logits and writing the gradient (8 bytes an element); small batches by
// launches.  Three launches: k_balance_count leaves per-block histograms, k_balance adds them up
// (every block for itself, behind the loads of its first logits), walks the logits and leaves the
// column sums of its blocks, k_balance_finish adds those in block order.  A last block that did the
// last step behind an agent-scope fence instead took 72 us at T 16384, E 64: every block's fence wrote
// the L2's whole share of the gradient back.  Few elements take one launch of one block, which counts
// and finishes for itself.  Column sums are fp32 inside a block (256 blocks share the tokens: 256
// experts' 8 million tokens are 512 additions a lane) and fp64 across blocks; the loss is evaluated
// in fp64.  T 16384, E 64, top-6: 3.2 + 8.2 + 3.8 us; T 32771, E 256, top-8 (67 MB): 4.7 + 20.6 + 7.2.  Of
// the 20.6, adding up 64 histograms in every block instead of one takes 1.5 (16 histograms: 18.7, but
// k_balance_count 9.4); 64 blocks instead of 256 make the last launch 4.7 and the pass 32.
#include "router_rows.h"

namespace moe {

namespace {

constexpr int kCountCopies = 8;
constexpr int kThreads = 1024;
constexpr int kMaxCountBlocks = 64, kMaxBlocks = 256;
// Up to this many logits one block does everything (one block / three launches, us: E 8, T 2048 11.2 /
// 12.2, T 4096 15.7 / 12.6; E 64, T 256 11.6 / 12.4, T 512 15.9 / 12.6).
constexpr int64_t kOneBlockElems = 16384;

// Histogram of the ids of valid tokens t0 .. t1 - 1 into hist[copy * (E + 1) + e] and their number
// into entry E; ids outside [0, E) are not counted.  hist is zero before; the caller syncs after.
// Four ids a thread are loaded before the first is counted.
__device__ __forceinline__ void count_tokens(const int32_t* __restrict__ ids,
                                             const uint8_t* __restrict__ mask, int64_t t0,
                                             int64_t t1, int E, int k, int* hist) {
  int* mine = hist + (threadIdx.x & (kCountCopies - 1)) * (E + 1);
  if (mask) {
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kThreads)
      if (mask[t]) atomicAdd(&mine[E], 1);
  } else if (threadIdx.x == 0 && t1 > t0) {
    mine[E] = (int)(t1 - t0);
  }
  const int32_t* base = ids + t0 * k;
  const uint32_t n = t1 > t0 ? (uint32_t)((t1 - t0) * k) : 0u;  // T k < 2^31
  for (uint32_t i = threadIdx.x; i < n; i += 4 * kThreads) {
    int id[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = i + j * kThreads;
      id[j] = -1;
      if (at < n) id[j] = base[at];
      if (mask && at < n && !mask[t0 + at / (uint32_t)k]) id[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((unsigned)id[j] < (unsigned)E) atomicAdd(&mine[id[j]], 1);
  }
}

// part[b * (E + 1) + e]: block b's histogram (entry E: its valid tokens)
__global__ __launch_bounds__(kThreads) void k_balance_count(
    const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int64_t T, int E, int k,
    int64_t per_block, int* __restrict__ part) {
  __shared__ int hist[kCountCopies * 257];
  for (int i = threadIdx.x; i < kCountCopies * (E + 1); i += kThreads) hist[i] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * per_block, t1 = t0 + per_block < T ? t0 + per_block : T;
  count_tokens(ids, mask, t0, t1, E, k, hist);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kThreads) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < kCountCopies; ++j) c += hist[j * (E + 1) + e];
    part[(int64_t)blockIdx.x * (E + 1) + e] = c;
  }
}

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  int64_t T;
  int E, k;
  double coef, grad_scale;
  const int* count_part;  // histograms of k_balance_count, or NULL: this block counts
  int count_blocks;
  int blocks;       // of k_balance
  float* sum_part;  // [blocks, E]
  int* totals;      // [E + 1]: the counts and the valid tokens, for k_balance_finish
  float *loss, *probs, *dlogits;  // probs, dlogits may be NULL
  int32_t* counts;                // may be NULL
};

__device__ __forceinline__ double balance_norm(const BalanceArgs& a, int64_t n) {
  return n > 0 ? a.coef * a.E / ((double)n * a.k) / (double)n : 0.0;
}

// The loss, the mean probabilities and the counts from column sums part [blocks][E] (all
// threads call; fin: kThreads doubles).  EG threads a row of sums, kThreads / EG rows at a time.
__device__ __forceinline__ void finish(const BalanceArgs& a, const float* part, int blocks,
                                       const int* cnt, double* fin) {
  const int tid = threadIdx.x, E = a.E;
  int EG = 1;
  while (EG < E) EG <<= 1;
  const int e = tid % EG, r0 = tid / EG, rows = kThreads / EG;
  double s = 0.0;
  if (e < E) {
    for (int b = r0; b < blocks; b += 16 * rows) {
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int at = b + j * rows;
        v[j] = 0.0f;
        if (at < blocks) v[j] = part[(int64_t)at * E + e];
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) s += (double)v[j];
    }
  }
  fin[tid] = s;
  __syncthreads();
  const int64_t n = cnt[E];
  double term = 0.0;
  if (tid < E) {
    s = 0.0;
    for (int r = 0; r < rows; ++r) s += fin[r * EG + tid];
    term = s * (double)cnt[tid];
    if (a.probs) a.probs[tid] = n > 0 ? (float)(s / (double)n) : 0.0f;
    if (a.counts) a.counts[tid] = cnt[tid];
  }
  __syncthreads();
  fin[tid] = term;
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (tid < o) fin[tid] += fin[tid + o];
  }
  if (tid == 0) *a.loss = (float)(balance_norm(a, n) * fin[0]);
}

__global__ __launch_bounds__(kThreads) void k_balance_finish(BalanceArgs a) {
  __shared__ double fin[kThreads];
  __shared__ int cnt[257];
  if ((int)threadIdx.x <= a.E) cnt[threadIdx.x] = a.totals[threadIdx.x];
  finish(a, a.sum_part, a.blocks, cnt, fin);  // syncs before it reads cnt
}

template <typename Row>
__global__ __launch_bounds__(kThreads) void k_balance(BalanceArgs a) {
  constexpr int LPT = Row::LPT, NV = Row::NV, TPW = Row::TPW, NW = kThreads / 64;
  __shared__ int cnt[257];
  __shared__ int hist[kCountCopies * 257];
  __shared__ float red[NW * 256];
  __shared__ double fin[kThreads];
  __shared__ int cmin;
  const int E = a.E, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane % LPT;

  // ---- the first tokens' logits on their way
  const int64_t step = (int64_t)gridDim.x * NW * TPW;
  int64_t t = ((int64_t)blockIdx.x * NW + wave) * TPW + lane / LPT;
  float next[NV];
  bool valid = false;
  auto load = [&](int64_t at) {
    valid = at < a.T && (!a.mask || a.mask[at]);
#pragma unroll
    for (int i = 0; i < NV; ++i) next[i] = -INFINITY;  // not valid: probabilities 0
    if (valid) Row::load(a.logits + at * E, E, l, -INFINITY, next);
  };
  load(t);

  // ---- counts, valid tokens and the smallest count
  if (tid == 0) cmin = 0x7FFFFFFF;
  if (tid <= E) cnt[tid] = 0;
  if (!a.count_part)
    for (int i = tid; i < kCountCopies * (E + 1); i += kThreads) hist[i] = 0;
  __syncthreads();
  if (a.count_part) {
    // all blocks' histograms, flat: entry i belongs to expert i % (E + 1)
    const int n = a.count_blocks * (E + 1), hop = kThreads % (E + 1);
    int e = tid % (E + 1);
    for (int i = tid; i < n; i += 8 * kThreads) {
      int c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = i + j * kThreads;
        c[j] = 0;
        if (at < n) c[j] = a.count_part[at];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (c[j]) atomicAdd(&cnt[e], c[j]);
        e += hop;
        if (e > E) e -= E + 1;
      }
    }
  } else {
    count_tokens(a.ids, a.mask, 0, a.T, E, a.k, hist);
    __syncthreads();
    if (tid <= E) {
      int c = 0;
#pragma unroll
      for (int j = 0; j < kCountCopies; ++j) c += hist[j * (E + 1) + tid];
      cnt[tid] = c;
    }
  }
  __syncthreads();
  if (tid < E) atomicMin(&cmin, cnt[tid]);
  __syncthreads();
  if (a.count_part && blockIdx.x == 0 && tid <= E) a.totals[tid] = cnt[tid];
  // The gradient's factor as mantissa and exponent: coef and grad_scale are any fp32 numbers, and a
  // factor that left fp32 would make NaN of the zeros it multiplies (padding, equal counts).
  int gexp;
  const float gman = (float)frexp(a.grad_scale * balance_norm(a, cnt[E]), &gexp);
  float c[NV], acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = Row::expert(l, i);
    c[i] = e < E ? (float)(cnt[e] - cmin) : 0.0f;
    acc[i] = 0.0f;
  }

  // ---- one pass over the logits (t - lane / LPT is the wave's first token of the step)
  for (; t - lane / LPT < a.T; t += step) {
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = next[i];
    load(t + step);
    Row::softmax(v);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      acc[i] += v[i];
      dot += v[i] * c[i];
    }
    if (a.dlogits) {
      dot = row_sum<LPT>(dot);
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = ldexpf(gman * v[i] * (c[i] - dot), gexp);
      if (t < a.T) Row::store(a.dlogits + t * E, E, l, v);
    }
  }

  // ---- column sums of the block
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int s = LPT; s < 64; s <<= 1) acc[i] += __shfl_xor(acc[i], s, 64);
    if (lane < LPT) {
      const int e = Row::expert(l, i);
      if (e < E) red[wave * 256 + e] = acc[i];
    }
  }
  __syncthreads();
  if (tid < E) {
    float s = 0.0f;
    for (int w = 0; w < NW; ++w) s += red[w * 256 + tid];
    if (a.count_part)
      a.sum_part[(int64_t)blockIdx.x * E + tid] = s;
    else
      red[tid] = s;
  }

  if (a.count_part) return;
  __syncthreads();
  finish(a, red, 1, cnt, fin);
}

int64_t count_blocks(const moe_shape& s) {
  const int64_t b = (s.T * s.top_k + 4095) / 4096;
  return b < 1 ? 1 : b > kMaxCountBlocks ? kMaxCountBlocks : b;
}

}  // namespace

// Workspace: the totals, the histograms and the column sums of the blocks.
size_t balance_ws_bytes(const moe_shape& s) {
  size_t o = 2048;
  o += ((size_t)kMaxCountBlocks * (s.n_experts + 1) * 4 + 255) & ~(size_t)255;
  o += ((size_t)kMaxBlocks * s.n_experts * 4 + 255) & ~(size_t)255;
  return o;
}

hipError_t launch_balance(const moe_shape& s, const float* logits, const int32_t* ids,
                          const uint8_t* mask, float coef, float grad_scale, float* loss,
                          int32_t* counts, float* probs, float* dlogits, void* ws,
                          hipStream_t st) {
  const int E = s.n_experts;
  BalanceArgs a = {};
  a.logits = logits;
  a.ids = ids;
  a.mask = mask;
  a.T = s.T;
  a.E = E;
  a.k = s.top_k;
  a.coef = coef;
  a.grad_scale = grad_scale;
  a.loss = loss;
  a.probs = probs;
  a.dlogits = dlogits;
  a.counts = counts;
  char* w = static_cast<char*>(ws);
  a.totals = reinterpret_cast<int*>(w);
  int* part = reinterpret_cast<int*>(w + 2048);
  a.sum_part = reinterpret_cast<float*>(
      w + 2048 + (((size_t)kMaxCountBlocks * (E + 1) * 4 + 255) & ~(size_t)255));
  const bool one = s.T * E <= kOneBlockElems && s.T * s.top_k <= kOneBlockElems;
  if (!one) {
    const int64_t nb = count_blocks(s), per = (s.T + nb - 1) / nb;
    hipLaunchKernelGGL(k_balance_count, dim3((unsigned)nb), dim3(kThreads), 0, st, ids, mask,
                       s.T, E, s.top_k, per, part);
    if (hipError_t err = hipGetLastError(); err != hipSuccess) return err;
    a.count_part = part;
    a.count_blocks = (int)nb;
  }
  const bool vec = E % 4 == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)dlogits % 16 == 0;
  return with_router_row(E, vec, [&](auto row) {
    using Row = decltype(row);
    const int64_t tokens = kThreads / 64 * Row::TPW;  // a block's tokens at a time
    int64_t blocks = (s.T + tokens - 1) / tokens;
    blocks = one ? 1 : blocks < kMaxBlocks ? blocks : kMaxBlocks;
    a.blocks = (int)blocks;
    hipLaunchKernelGGL(k_balance<Row>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
    if (hipError_t err = hipGetLastError(); err != hipSuccess || one) return err;
    hipLaunchKernelGGL(k_balance_finish, dim3(1), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  });
}

}  // namespace moe
