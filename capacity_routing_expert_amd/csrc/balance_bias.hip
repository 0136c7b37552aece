// Update of the selection bias: experts that got more than their even share of the assignments are
// chosen a little less from now on, the others a little more.
//
//   total = sum of c_e over the experts that are on (bias not -inf), n of them
//   bias_e += rate sign(total - n c_e)
// The comparison is in whole numbers.  Two launches, histograms of token ranges and their sum; few
// assignments, or counts that are given, take the second alone.
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 1024;
constexpr int kCopies = 8;  // histograms a block, so that neighbouring lanes seldom meet at one counter
constexpr int kMaxBlocks = 64;
constexpr int64_t kOneBlock = 16384;  // assignments that one block counts by itself

int64_t count_blocks(int64_t n) {
  if (n <= kOneBlock) return 0;
  const int64_t b = (n + 4095) / 4096;
  return b < kMaxBlocks ? b : kMaxBlocks;
}

// Histogram of assignments i0 .. i1 - 1 of valid tokens into hist (zero before): ids outside [0, E)
// are not counted.
__device__ __forceinline__ void count_range(const int32_t* __restrict__ ids,
                                            const uint8_t* __restrict__ mask, int64_t i0,
                                            int64_t i1, int E, int k, int* hist) {
  int* mine = hist + (threadIdx.x & (kCopies - 1)) * (E + 1);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += 4 * kThreads) {
    int id[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = i + j * kThreads;
      id[j] = at < i1 ? ids[at] : -1;
      if (mask && at < i1 && !mask[(uint32_t)at / (uint32_t)k]) id[j] = -1;  // T k < 2^31
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((unsigned)id[j] < (unsigned)E) atomicAdd(&mine[id[j]], 1);
  }
}

__global__ __launch_bounds__(kThreads) void k_bias_count(const int32_t* __restrict__ ids,
                                                         const uint8_t* __restrict__ mask,
                                                         int64_t n, int E, int k,
                                                         int64_t per_block, int* __restrict__ part) {
  __shared__ int hist[kCopies * 257];
  for (int i = threadIdx.x; i < kCopies * (E + 1); i += kThreads) hist[i] = 0;
  __syncthreads();
  const int64_t i0 = blockIdx.x * per_block, i1 = i0 + per_block < n ? i0 + per_block : n;
  count_range(ids, mask, i0, i1, E, k, hist);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < kCopies; ++j) c += hist[j * (E + 1) + e];
    part[(int64_t)blockIdx.x * E + e] = c;
  }
}

// blocks > 0: the counts are the sums of part; otherwise ids, if given, are counted here; otherwise
// counts holds them.
__global__ __launch_bounds__(kThreads) void k_bias_update(const int32_t* __restrict__ ids,
                                                          const uint8_t* __restrict__ mask,
                                                          int64_t n, int E, int k,
                                                          const int* __restrict__ part, int blocks,
                                                          float rate, float* __restrict__ bias,
                                                          int32_t* __restrict__ counts) {
  __shared__ int hist[kCopies * 257];
  __shared__ long long total;
  __shared__ int on;
  for (int i = threadIdx.x; i < kCopies * (E + 1); i += kThreads) hist[i] = 0;
  if (threadIdx.x == 0) {
    total = 0;
    on = 0;
  }
  __syncthreads();
  if (blocks > 0) {
    // EG threads a row of partial counts, kThreads / EG rows at a time, their loads together
    int EG = 1;
    while (EG < E) EG <<= 1;
    const int at = threadIdx.x % EG, r0 = threadIdx.x / EG, rows = kThreads / EG;
    if (at < E)
      for (int b = r0; b < blocks; b += 16 * rows) {
        int v[16], c = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = part[(b + j * rows < blocks ? b + j * rows : b) * E + at];
#pragma unroll
        for (int j = 0; j < 16; ++j) c += b + j * rows < blocks ? v[j] : 0;
        atomicAdd(&hist[(r0 & (kCopies - 1)) * (E + 1) + at], c);
      }
  } else if (ids) {
    count_range(ids, mask, 0, n, E, k, hist);
  }
  __syncthreads();
  const int e = threadIdx.x;
  int c = 0;
  float b = 0.0f;
  if (e < E) {
    if (blocks > 0 || ids) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) c += hist[j * (E + 1) + e];
      if (counts) counts[e] = c;
    } else {
      c = counts[e];
    }
    b = bias[e];
    if (b != -INFINITY) {
      atomicAdd((unsigned long long*)&total, (unsigned long long)(long long)c);
      atomicAdd(&on, 1);
    }
  }
  __syncthreads();
  if (e < E && b != -INFINITY) {
    const long long over = total - (long long)on * c;
    bias[e] = over > 0 ? b + rate : over < 0 ? b - rate : b;
  }
}

}  // namespace

size_t balance_bias_ws_bytes(const moe_shape& s) {
  const int64_t b = count_blocks(s.T * (int64_t)s.top_k);
  return ((size_t)b * s.n_experts * 4 + 255) & ~(size_t)255;
}

hipError_t launch_balance_bias(const moe_shape& s, const int32_t* ids, const uint8_t* mask,
                               float rate, float* bias, int32_t* counts, void* ws,
                               hipStream_t st) {
  const int64_t n = s.T * (int64_t)s.top_k;
  const int blocks = ids ? (int)count_blocks(n) : 0;
  if (blocks > 0) {
    const int64_t per = (n + blocks - 1) / blocks;
    hipLaunchKernelGGL(k_bias_count, dim3(blocks), dim3(kThreads), 0, st, ids, mask, n, s.n_experts,
                       s.top_k, per, (int*)ws);
    if (hipError_t err = hipGetLastError(); err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(k_bias_update, dim3(1), dim3(kThreads), 0, st, ids, mask, n, s.n_experts,
                     s.top_k, (const int*)ws, blocks, rate, bias, counts);
  return hipGetLastError();
}

}  // namespace moe
