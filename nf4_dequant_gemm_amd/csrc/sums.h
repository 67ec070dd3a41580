// Sums of float32 partials in a fixed order (lora.hip, thin.hip).
#pragma once

#include "common.h"

namespace nf4q {

// The sum of `splits` partials [r][C] at p, four consecutive outputs, in a fixed order (loads issued eight at a time).
__device__ __forceinline__ f32x4 split_sum4(const float *p, int64_t n, int splits) {
  f32x4 a = {0.f, 0.f, 0.f, 0.f};
  for (int sp = 0; sp < splits; sp += 8) {
    f32x4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (sp + j < splits) v[j] = *reinterpret_cast<const f32x4 *>(p + (int64_t)(sp + j) * n);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (sp + j < splits) a += v[j];
  }
  return a;
}

// The sum of `splits` partials at p, n apart, sequential, loads issued eight at a time.
__device__ __forceinline__ float split_sum1(const float *p, int64_t n, int splits) {
  float a = 0.f;
  int s = 0;
  for (; s + 8 <= splits; s += 8) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p[(int64_t)(s + j) * n];
#pragma unroll
    for (int j = 0; j < 8; ++j) a += v[j];
  }
  for (; s < splits; ++s) a += p[(int64_t)s * n];
  return a;
}

// out[i] (bf16) and wide[i] (float32; NULL: none) = the sum of `splits` partials [n] at part; workgroup `block` of
// `blocks`.
__device__ __forceinline__ void split_sum_each(const float *__restrict__ part, int64_t n, int splits,
                                               uint16_t *__restrict__ out, float *__restrict__ wide, int64_t block,
                                               int64_t blocks) {
  for (int64_t i = block * blockDim.x + threadIdx.x; i < n; i += blocks * blockDim.x) {
    const float a = split_sum1(part + i, n, splits);
    out[i] = (uint16_t)(pack_bf16x2(a, 0.f) & 0xFFFFu);
    if (wide) wide[i] = a;
  }
}

// out[c][j] (bf16, contiguous) = s * the sum of `splits` partials [r][C] at part, for the 64 columns from c0 on
// and all r <= 128 ranks, through LDS: the outputs of 64 columns are contiguous (written one by one at a stride of
// r they took 9.1 us at r 64, C 11008, now 4.8). C % 8 == 0; split_sum_t_threads(r) threads, 16 for each rank up to 1024.
__device__ __forceinline__ void split_sum_t(const float *__restrict__ part, int64_t C, int r, int splits, float s,
                                            uint16_t *__restrict__ out, int64_t c0) {
  __shared__ uint16_t tile[64 * 129];       // [column][rank], rows of an odd length: columns in different banks
  const int64_t n = (int64_t)r * C;
  const int c = (threadIdx.x & 15) * 4, cols = C - c0 < 64 ? (int)(C - c0) : 64, row = r | 1;
  const float *p = part + c0 + c;
  for (int j = threadIdx.x >> 4; j < r; j += blockDim.x >> 4) {
    if (c >= cols) continue;
    const f32x4 a = split_sum4(p + (int64_t)j * C, n, splits);
#pragma unroll
    for (int e = 0; e < 4; ++e) tile[(c + e) * row + j] = (uint16_t)(pack_bf16x2(s * a[e], 0.f) & 0xFFFFu);
  }
  __syncthreads();
  uint16_t *o = out + c0 * r;
  for (int i = threadIdx.x; i < cols * r / 8; i += blockDim.x) {      // cols is a multiple of 8
    int at = 8 * i / r * row + 8 * i % r, left = r - 8 * i % r;
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = tile[at];
      v[e / 2] = e & 1 ? v[e / 2] | (h << 16) : h;
      ++at;
      if (--left == 0) {
        at += row - r;
        left = r;
      }
    }
    *reinterpret_cast<u32x4 *>(o + 8 * i) = v;
  }
}
inline int split_sum_t_threads(int r) { return r > 32 ? 1024 : r > 16 ? 512 : 256; }

}  // namespace nf4q
