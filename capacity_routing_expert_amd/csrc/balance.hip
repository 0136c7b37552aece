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
// launches.  Two launches: k_balance_count leaves per-block histograms, k_balance walks the
// logits and its last block (a ticket that k_balance_count zeroed) adds the blocks' column sums
// in block order, so no result depends on the order of arrival.  Few elements take one launch of
// one block, which counts for itself.  Column sums are fp32 inside a block (at most some hundred
// tokens a lane) and fp64 across blocks; the loss is evaluated in fp64.
#include "router_rows.h"

namespace moe {

namespace {

constexpr int kCountThreads = 256, kCountCopies = 8;
constexpr int kThreads = 512;
constexpr int kMaxCountBlocks = 64, kMaxBlocks = 256;
// Up to this many logits one block does everything.
constexpr int64_t kOneBlockElems = 8192;

// Histogram of the ids of valid tokens t0 .. t1 - 1 into hist[copy * (E + 1) + e] and their number
// into entry E; ids outside [0, E) are not counted.  hist is zero before; the caller syncs after.
__device__ __forceinline__ void count_tokens(const int32_t* __restrict__ ids,
                                             const uint8_t* __restrict__ mask, int64_t t0,
                                             int64_t t1, int E, int k, int* hist) {
  int* mine = hist + (threadIdx.x & (kCountCopies - 1)) * (E + 1);
  for (int64_t t = t0 + threadIdx.x; t < t1; t += blockDim.x)
    if (!mask || mask[t]) atomicAdd(&mine[E], 1);
  const int64_t end = t1 * k;
  for (int64_t i = t0 * k + threadIdx.x; i < end; i += blockDim.x) {
    const int id = ids[i];
    if ((unsigned)id < (unsigned)E && (!mask || mask[i / k])) atomicAdd(&mine[id], 1);
  }
}

// part[b * (E + 1) + e]: block b's histogram (entry E: its valid tokens); *ticket = 0
__global__ __launch_bounds__(kCountThreads) void k_balance_count(
    const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int64_t T, int E, int k,
    int64_t per_block, int* __restrict__ part, int* __restrict__ ticket) {
  __shared__ int hist[kCountCopies * 257];
  for (int i = threadIdx.x; i < kCountCopies * (E + 1); i += kCountThreads) hist[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * per_block, t1 = t0 + per_block < T ? t0 + per_block : T;
  count_tokens(ids, mask, t0, t1, E, k, hist);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kCountThreads) {
    int c = 0;
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
  float* sum_part;  // [blocks, E]
  int* ticket;
  float *loss, *probs, *dlogits;  // probs, dlogits may be NULL
  int32_t* counts;                // may be NULL
};

template <typename Row>
__global__ __launch_bounds__(kThreads) void k_balance(BalanceArgs a) {
  constexpr int LPT = Row::LPT, NV = Row::NV, TPW = Row::TPW, NW = kThreads / 64;
  __shared__ int cnt[257];
  __shared__ int hist[kCountCopies * 257];
  __shared__ float red[NW * 256];
  __shared__ double fin[kThreads];
  __shared__ int cmin, last;
  const int E = a.E, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane % LPT;

  // ---- counts, valid tokens and the smallest count
  if (!a.count_part) {
    for (int i = tid; i < kCountCopies * (E + 1); i += kThreads) hist[i] = 0;
    __syncthreads();
    count_tokens(a.ids, a.mask, 0, a.T, E, a.k, hist);
  }
  if (tid == 0) cmin = 0x7FFFFFFF;
  __syncthreads();
  if (tid <= E) {
    int c = 0;
    if (a.count_part) {
      for (int b = 0; b < a.count_blocks; ++b) c += a.count_part[(int64_t)b * (E + 1) + tid];
    } else {
      for (int j = 0; j < kCountCopies; ++j) c += hist[j * (E + 1) + tid];
    }
    cnt[tid] = c;
    if (tid < E) atomicMin(&cmin, c);
  }
  __syncthreads();
  const int64_t n = cnt[E];
  const double norm = n > 0 ? a.coef * E / ((double)n * a.k) / (double)n : 0.0;
  const float gscale = (float)(a.grad_scale * norm);
  float c[NV], acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = Row::expert(l, i);
    c[i] = e < E ? (float)(cnt[e] - cmin) : 0.0f;
    acc[i] = 0.0f;
  }

  // ---- one pass over the logits
  const int64_t step = (int64_t)gridDim.x * NW * TPW;
  for (int64_t t0 = ((int64_t)blockIdx.x * NW + wave) * TPW; t0 < a.T; t0 += step) {
    const int64_t t = t0 + lane / LPT;
    const bool in = t < a.T, valid = in && (!a.mask || a.mask[t]);
    float v[NV];
    if (valid) {
      Row::load(a.logits + t * E, E, l, -INFINITY, v);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = -INFINITY;  // probabilities 0
    }
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
      for (int i = 0; i < NV; ++i) v[i] = gscale * v[i] * (c[i] - dot);
      if (in) Row::store(a.dlogits + t * E, E, l, v);
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

  // ---- the last block: S, the loss and the counts
  int blocks = 1;
  if (a.count_part) {
    blocks = gridDim.x;
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(a.ticket, 1) == blocks - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
  } else {
    __syncthreads();
  }
  // EG threads a row of partial sums, kThreads / EG rows at a time
  int EG = 1;
  while (EG < E) EG <<= 1;
  const int e = tid % EG, r0 = tid / EG, rows = kThreads / EG;
  double s = 0.0;
  if (e < E) {
    if (a.count_part) {
#pragma unroll 16
      for (int b = r0; b < blocks; b += rows) s += (double)a.sum_part[(int64_t)b * E + e];
    } else if (r0 == 0) {
      s = (double)red[e];
    }
  }
  fin[tid] = s;
  __syncthreads();
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
  if (tid == 0) *a.loss = (float)(norm * fin[0]);
}

int64_t count_blocks(const moe_shape& s) {
  const int64_t b = (s.T * s.top_k + 4095) / 4096;
  return b < 1 ? 1 : b > kMaxCountBlocks ? kMaxCountBlocks : b;
}

}  // namespace

// Workspace: [0] the ticket, then the histograms and the column sums of the blocks.
size_t balance_ws_bytes(const moe_shape& s) {
  size_t o = 256;
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
  a.ticket = reinterpret_cast<int*>(w);
  int* part = reinterpret_cast<int*>(w + 256);
  a.sum_part = reinterpret_cast<float*>(
      w + 256 + (((size_t)kMaxCountBlocks * (E + 1) * 4 + 255) & ~(size_t)255));
  const bool one = s.T * E <= kOneBlockElems && s.T * s.top_k <= kOneBlockElems;
  if (!one) {
    const int64_t nb = count_blocks(s), per = (s.T + nb - 1) / nb;
    hipLaunchKernelGGL(k_balance_count, dim3((unsigned)nb), dim3(kCountThreads), 0, st, ids, mask,
                       s.T, E, s.top_k, per, part, a.ticket);
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
    hipLaunchKernelGGL(k_balance<Row>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  });
}

}  // namespace moe
