// Expert weights at 4 bits: quantising, and reading back.
//
// Code: a sign bit and three bits of magnitude, {0, 0.5, 1, 1.5, 2, 3, 4, 6} (2 exponent bits, 1
// mantissa bit): the 4-bit format that gfx950 converts to bf16 pairs in one instruction
// (v_cvt_scalef32_pk_bf16_fp4), so the products spend half an instruction a weight on it.  One
// bf16 scale per `group` consecutive columns of a row: s = max|w| / 6 (the largest magnitude),
// w ~ s * value(code).
//
// Codes are stored in the order that the products read: blocks of 8 rows x 128 columns, 512
// bytes each, [E][ceil(cols / 128)][rows / 8]; in a block, 16 bytes belong to row r and the
// column octets o, o + 4, o + 8, o + 12 (o = 0 .. 3), at (8 o + r) 16, a dword an octet, its
// first column in the lowest 4 bits.  So the 64 lanes of a wave that feed 16 rows x 32 columns
// per matrix instruction read two whole blocks, 16 bytes a lane, for four instructions, and the
// waves of a workgroup, on neighbouring rows of the same columns, one run of memory.  Scales:
// [E][ceil(cols / 128)][rows][128 / group], the ones past cols zero.
//
// Bound: HBM (2 or 4 bytes in, 0.5 + 2 / group out, a weight) and, short of it, the division.  A wave
// takes one block; a lane 16 columns of a row, so a group is 2, 4 or 8 lanes.  8 x 8192 x 2048 bf16
// weights, group 32 (268 MB in, 75 MB out): 127 - 145 us, 2.4 - 2.7 TB/s; with a product by the scale's
// reciprocal instead of the division 113 (not the same codes), with stores of whole runs no less.
// Reading back (75 MB in, 537 MB out): 328 us, 1.9 TB/s, eight 4-byte stores a lane, as w lies on 4 bytes.
#include "moe_internal.h"

namespace moe {

namespace {

// magnitude code of a >= 0: the nearest magnitude, ties to the even code
__device__ __forceinline__ uint32_t magnitude_code(float a) {
  return (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
         (a > 5.0f);
}

template <typename TIn>
__device__ __forceinline__ void load8(const TIn* p, float* v) {
  if constexpr (sizeof(TIn) == 2) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i];
  }
}

template <typename TIn>
__global__ __launch_bounds__(256) void k_quantize(const TIn* __restrict__ w,
                                                  uint32_t* __restrict__ codes,
                                                  bf16_t* __restrict__ scales, int64_t blocks,
                                                  int rows, int cols, int KC, int group) {
  const int lane = threadIdx.x & 63, r = lane & 7, kg = lane >> 3;
  const int per = 128 / group;  // groups of a block of columns
  for (int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); b < blocks;
       b += (int64_t)gridDim.x * 4) {
    const int r8 = (int)(b % (rows / 8)), kc = (int)(b / (rows / 8) % KC);  // block [e][kc][r8]
    const int64_t row = b / (rows / 8) / KC * rows + r8 * 8 + r;
    const int c0 = kc * 128 + kg * 16;
    float v[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (c0 + 8 * h < cols) {
        load8(w + row * cols + c0 + 8 * h, v + 8 * h);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] = 0.0f;
      }
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
    for (int s = 8; s < group / 2; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
    const bf16_t sb = f32_to_bf16(m * (1.0f / 6.0f));
    const float s = bf16_to_f32(sb);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = v[8 * h + i];
        const uint32_t code = (s > 0.0f ? magnitude_code(fabsf(x) / s) : 0u) |
                              (__float_as_uint(x) >> 31 << 3);
        word |= code << (4 * i);
      }
      // column octet kg * 2 + h of the block: dword (octet / 4) of unit (octet % 4)
      const int oct = kg * 2 + h;
      codes[b * 128 + ((oct & 3) * 8 + r) * 4 + (oct >> 2)] = word;
    }
    if (kg * 16 % group == 0) scales[(b * 8 + r) * per + kg * 16 / group] = sb;
  }
}

// One thread an octet of columns.
__global__ __launch_bounds__(256) void k_dequantize(const uint32_t* __restrict__ codes,
                                                    const bf16_t* __restrict__ scales,
                                                    float* __restrict__ w, int64_t all_rows,
                                                    int rows, int cols, int KC, int group) {
  const int per = 128 / group, octs = cols / 8;
  const int64_t n = all_rows * octs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / octs;
    const int c = (int)(i % octs) * 8, kc = c / 128, oct = c % 128 / 8;
    const int64_t at = (row / rows * KC + kc) * rows + row % rows;  // [e][kc][row]
    const uint32_t word = codes[at / 8 * 128 + ((oct & 3) * 8 + at % 8) * 4 + (oct >> 2)];
    const float s = bf16_to_f32(scales[at * per + oct * 8 / group]);
    float* o = w + row * cols + c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t q = word >> (4 * j), e = q >> 1 & 3, m = q & 1;
      // exponent 0: m / 2; else (1 + m / 2) 2^(e - 1)
      const float mag = e == 0 ? 0.5f * m : (1.0f + 0.5f * m) * (float)(1 << (e - 1));
      o[j] = (q & 8 ? -mag : mag) * s;
    }
  }
}

}  // namespace

int64_t quantized_codes_bytes(int64_t E, int rows, int cols) {
  return E * rows * (((int64_t)cols + 127) / 128) * 64;
}
int64_t quantized_scales_count(int64_t E, int rows, int cols, int group) {
  return E * rows * (((int64_t)cols + 127) / 128) * (128 / group);
}

hipError_t launch_quantize(const void* w, bool bf16, int64_t E, int rows, int cols, int group,
                           void* codes, void* scales, hipStream_t st) {
  const int KC = (cols + 127) / 128;
  const int64_t blocks = E * (rows / 8) * KC, wg = (blocks + 3) / 4;
  const dim3 grid((unsigned)(wg < 65536 ? wg : 65536));
  if (bf16)
    hipLaunchKernelGGL(k_quantize<bf16_t>, grid, dim3(256), 0, st, (const bf16_t*)w,
                       (uint32_t*)codes, (bf16_t*)scales, blocks, rows, cols, KC, group);
  else
    hipLaunchKernelGGL(k_quantize<float>, grid, dim3(256), 0, st, (const float*)w,
                       (uint32_t*)codes, (bf16_t*)scales, blocks, rows, cols, KC, group);
  return hipGetLastError();
}

hipError_t launch_dequantize(const void* codes, const void* scales, int64_t E, int rows, int cols,
                             int group, float* w, hipStream_t st) {
  const int64_t n = E * rows * (cols / 8), blocks = (n + 255) / 256;
  hipLaunchKernelGGL(k_dequantize, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                     st, (const uint32_t*)codes, (const bf16_t*)scales, w, E * rows, rows, cols,
                     (cols + 127) / 128, group);
  return hipGetLastError();
}

}  // namespace moe
