// Tokens into expert order and the experts' outputs back, with their gradients (gfx950).
//
// place[i][j] is the row of token i's j-th choice among the grouped rows (-1: none), source[p] the token of
// row p (-1: a row behind the last). Over tokens i and choices j:
//
//   gather       G[place_ij] = X_i, rows without a token 0
//   combine      Y_i = base_i + sum_j gate_ij Z[place_ij]      (without gates: the gradient of gather)
//   combine_bwd  dZ[place_ij] = gate_ij dY_i,  dgate_ij = <dY_i, Z[place_ij]>,  rows without a token 0
//
// All three read and write each element once and are bound by memory, so each is organised by token:
// what belongs to the token (X, dY, the sum of Y) is read or written once, in registers meanwhile, and the
// rows of its choices are whole contiguous rows. Rows behind the last are zeroed by the token whose share
// of the row numbers they fall in. Elements move in 16-byte chunks where row starts allow it, else one by
// one. Sums are float32 in the order of the choices, rounded once.
#include "common.h"
#include "launch.h"

namespace nf4q {
namespace {

// A chunk of kP elements of type T (uint16_t: bf16, or float): 16 bytes, or one element.
template <typename T, bool kVec>
struct Chunk;
template <typename T>
struct Chunk<T, true> {
  static constexpr int P = 16 / (int)sizeof(T);
  u32x4 v;
  __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const u32x4 *>(p); }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<u32x4 *>(p) = v; }
  __device__ __forceinline__ void zero() { v = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 2) return (e & 1) ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]);
    else return __uint_as_float(v[e]);
  }
  __device__ __forceinline__ void set(const float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      else v[i] = __float_as_uint(f[i]);
    }
  }
};
template <typename T>
struct Chunk<T, false> {
  static constexpr int P = 1;
  T v;
  __device__ __forceinline__ void load(const T *p) { v = *p; }
  __device__ __forceinline__ void store(T *p) const { *p = v; }
  __device__ __forceinline__ void zero() { v = 0; }
  __device__ __forceinline__ float get(int) const {
    if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
    else return v;
  }
  __device__ __forceinline__ void set(const float *f) {
    if constexpr (sizeof(T) == 2) v = (uint16_t)(pack_bf16x2(f[0], 0.f) & 0xFFFFu);
    else v = f[0];
  }
};

// The place of a choice, -1 where it is none (whatever it holds then).
__device__ __forceinline__ int64_t place_of(const MoeRowsArgs &a, int64_t i) {
  const int p = __builtin_amdgcn_readfirstlane(a.place[i]);
  return p >= 0 && p < a.t * a.top ? p : -1;
}
__device__ __forceinline__ bool no_token(const MoeRowsArgs &a, int64_t row) {
  const int s = __builtin_amdgcn_readfirstlane(a.source[row]);
  return s < 0 || s >= a.t;
}

// One wave: token `i`, chunks [seg * 64 U, ..) of its rows, U for each lane.
template <typename T, bool kVec, int U, bool kGather>
__global__ __launch_bounds__(256) void rows_kernel(MoeRowsArgs a, int64_t segs) {
  using C = Chunk<T, kVec>;
  const int lane = threadIdx.x & 63;
  const int64_t chunks = a.d / C::P, waves = (int64_t)gridDim.x * 4;
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < a.t * segs; w += waves) {
    const int64_t i = w / segs, c0 = (w - i * segs) * 64 * U + lane;
    if constexpr (kGather) {
      const T *x = reinterpret_cast<const T *>(a.x) + i * a.ldx;
      T *out = reinterpret_cast<T *>(a.out);
      C v[U], zero;
      zero.zero();
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + 64 * u < chunks) v[u].load(x + (c0 + 64 * u) * C::P);
      for (int j = 0; j < a.top; ++j) {
        const int64_t p = place_of(a, i * a.top + j);
        if (p >= 0) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c0 + 64 * u < chunks) v[u].store(out + p * a.d + (c0 + 64 * u) * C::P);
        }
        if (no_token(a, i * a.top + j)) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c0 + 64 * u < chunks) zero.store(out + (i * a.top + j) * a.d + (c0 + 64 * u) * C::P);
        }
      }
    } else {
      const T *z = reinterpret_cast<const T *>(a.x);
      T *y = reinterpret_cast<T *>(a.out) + i * a.ldo;
      float acc[U][C::P];
      C b[U];
      if (a.base) {
        const T *base = reinterpret_cast<const T *>(a.base) + i * a.ldb;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c0 + 64 * u < chunks) b[u].load(base + (c0 + 64 * u) * C::P);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < C::P; ++e) acc[u][e] = a.base ? b[u].get(e) : 0.f;
      for (int j0 = 0; j0 < a.top; j0 += 4) {      // the rows of up to four choices requested together
        C v[4][U];
        float g[4];
        int64_t p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          p[k] = j0 + k < a.top ? place_of(a, i * a.top + j0 + k) : -1;
          if (p[k] >= 0) {
            g[k] = a.gate ? a.gate[i * a.top + j0 + k] : 1.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (c0 + 64 * u < chunks) v[k][u].load(z + p[k] * a.d + (c0 + 64 * u) * C::P);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (p[k] >= 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int e = 0; e < C::P; ++e) acc[u][e] += g[k] * v[k][u].get(e);
          }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + 64 * u < chunks) {
          C o;
          o.set(acc[u]);
          o.store(y + (c0 + 64 * u) * C::P);
        }
    }
  }
}

// One workgroup takes a token at a time: up to four choices in a pass over dY.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void rows_bwd_kernel(MoeRowsArgs a) {
  using C = Chunk<T, kVec>;
  __shared__ float s_dot[4][4];
  const int tid = threadIdx.x, waves = blockDim.x / 64;
  const int64_t chunks = a.d / C::P;
  const T *z = reinterpret_cast<const T *>(a.z);
  T *dz = reinterpret_cast<T *>(a.out);
  for (int64_t i = blockIdx.x; i < a.t; i += gridDim.x) {
    const T *dy = reinterpret_cast<const T *>(a.x) + i * a.ldx;
    for (int j0 = 0; j0 < a.top; j0 += 4) {
      int64_t p[4];
      float g[4], dot[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[k] = j0 + k < a.top ? place_of(a, i * a.top + j0 + k) : -1;
        g[k] = p[k] >= 0 ? a.gate[i * a.top + j0 + k] : 0.f;
        dot[k] = 0.f;
      }
      for (int64_t c = tid; c < chunks; c += blockDim.x) {
        C y, v[4], o;
        y.load(dy + c * C::P);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (p[k] >= 0) v[k].load(z + p[k] * a.d + c * C::P);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (p[k] >= 0) {
            float f[C::P];
#pragma unroll
            for (int e = 0; e < C::P; ++e) {
              dot[k] += y.get(e) * v[k].get(e);
              f[e] = g[k] * y.get(e);
            }
            o.set(f);
            o.store(dz + p[k] * a.d + c * C::P);
          }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        for (int s = 32; s; s >>= 1) dot[k] += __shfl_xor(dot[k], s);
        if ((tid & 63) == 0) s_dot[tid >> 6][k] = dot[k];
      }
      __syncthreads();
      if (tid < 4 && j0 + tid < a.top) {
        float sum = 0.f;
        for (int w = 0; w < waves; ++w) sum += s_dot[w][tid];
        a.dgate[i * a.top + j0 + tid] = sum;
      }
      __syncthreads();
    }
    for (int j = 0; j < a.top; ++j)
      if (no_token(a, i * a.top + j)) {
        C zero;
        zero.zero();
        for (int64_t c = tid; c < chunks; c += blockDim.x) zero.store(dz + (i * a.top + j) * a.d + c * C::P);
      }
  }
}

template <typename T, bool kVec, bool kGather>
hipError_t launch_rows_as(const MoeRowsArgs &a, hipStream_t st) {
  const int64_t chunks = a.d / Chunk<T, kVec>::P;
  constexpr int kWide = 4;
  // four chunks a lane once that still gives every CU 16 waves
  const int U = a.t * ((chunks + 64 * kWide - 1) / (64 * kWide)) >= 4096 ? kWide : 1;
  const int64_t segs = (chunks + 64 * U - 1) / (64 * U);
  int64_t blocks = (a.t * segs + 3) / 4;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  if (U == kWide)
    rows_kernel<T, kVec, kWide, kGather><<<dim3((unsigned)blocks), dim3(256), 0, st>>>(a, segs);
  else
    rows_kernel<T, kVec, 1, kGather><<<dim3((unsigned)blocks), dim3(256), 0, st>>>(a, segs);
  return hipGetLastError();
}

bool vec_rows(const MoeRowsArgs &a, size_t esz) {
  uintptr_t all = (uintptr_t)a.x | (uintptr_t)a.out | (uintptr_t)a.z | (uintptr_t)a.base;
  all |= (uintptr_t)((a.d | a.ldx | a.ldo | a.ldb) * (int64_t)esz);
  return (all & 15) == 0;
}

}  // namespace

hipError_t launch_gather(const MoeRowsArgs &a, bool f32, hipStream_t st) {
  if (vec_rows(a, f32 ? 4 : 2)) return f32 ? launch_rows_as<float, true, true>(a, st) : launch_rows_as<uint16_t, true, true>(a, st);
  return f32 ? launch_rows_as<float, false, true>(a, st) : launch_rows_as<uint16_t, false, true>(a, st);
}

hipError_t launch_combine(const MoeRowsArgs &a, bool f32, hipStream_t st) {
  if (vec_rows(a, f32 ? 4 : 2)) return f32 ? launch_rows_as<float, true, false>(a, st) : launch_rows_as<uint16_t, true, false>(a, st);
  return f32 ? launch_rows_as<float, false, false>(a, st) : launch_rows_as<uint16_t, false, false>(a, st);
}

hipError_t launch_combine_bwd(const MoeRowsArgs &a, bool f32, hipStream_t st) {
  const bool vec = vec_rows(a, f32 ? 4 : 2);
  const int64_t chunks = vec ? a.d / (f32 ? 4 : 8) : a.d;
  const unsigned threads = chunks <= 64 ? 64 : chunks <= 128 ? 128 : 256;
  const unsigned blocks = (unsigned)(a.t < (1 << 20) ? a.t : 1 << 20);
  if (vec) {
    if (f32) rows_bwd_kernel<float, true><<<dim3(blocks), dim3(threads), 0, st>>>(a);
    else rows_bwd_kernel<uint16_t, true><<<dim3(blocks), dim3(threads), 0, st>>>(a);
  } else {
    if (f32) rows_bwd_kernel<float, false><<<dim3(blocks), dim3(threads), 0, st>>>(a);
    else rows_bwd_kernel<uint16_t, false><<<dim3(blocks), dim3(threads), 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace nf4q
