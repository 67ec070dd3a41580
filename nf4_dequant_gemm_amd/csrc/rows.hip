// Tokens into expert order and the experts' outputs back, with their gradients (gfx950).
//
// place[i][j] is the row of token i's j-th choice among the grouped rows (-1: none), source[p] the token of
// row p (-1: a row behind the last). Over tokens i and choices j:
//
//   gather       G[place_ij] = X_i, rows without a token 0
//   combine      Y_i = base_i + sum_j gate_ij Z[place_ij]      (without gates: the gradient of gather)
//   combine_bwd  dZ[place_ij] = gate_ij dY_i,  dgate_ij = <dY_i, Z[place_ij]>,  rows without a token 0
//
// All three move each element once and are bound by memory, so each is organised by token: what belongs to the
// token (X, the sum of Y) is read or written once, in registers meanwhile (dY is read by a wave for each choice,
// neighbours that find it in the caches), and the rows of its choices are whole contiguous rows. Rows behind the
// last are zeroed by the token whose share of the row numbers they fall in. Elements move in 16-byte chunks, at
// any alignment of the rows. Sums are float32 in the order of the choices, rounded once.
//
// Measured on 8192 tokens of 4096 in bf16, two choices: gather 34.8 us and combine 42.4 us (201 MB each), the
// backward 57.7 us (335 MB), 4.7 to 5.8 TB/s; 1111 tokens of 1023 float32, six choices: 7.8, 7.8, 11.6 us.
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace nf4q {
namespace {

// A chunk of P elements of type T (uint16_t: bf16, or float): 16 bytes, aligned to 16 in memory (kAl) or to its
// elements, which the memory unit takes as well.
typedef u32x4 __attribute__((aligned(2))) u32x4_by2;
typedef u32x4 __attribute__((aligned(4))) u32x4_by4;
template <typename T, bool kAl>
struct Chunk {
  static constexpr int P = 16 / (int)sizeof(T);
  typedef std::conditional_t<kAl, u32x4, std::conditional_t<sizeof(T) == 2, u32x4_by2, u32x4_by4>> Mem;
  u32x4 v;
  __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const Mem *>(p); }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Mem *>(p) = v; }
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
__device__ __forceinline__ float value(T x) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(x);
  else return x;
}
template <typename T>
__device__ __forceinline__ T rounded(float x) {
  if constexpr (sizeof(T) == 2) return (uint16_t)(pack_bf16x2(x, 0.f) & 0xFFFFu);
  else return x;
}

// Up to 64 choices of a token at once, lane j holding choice j: one trip to memory for all of them.
struct Choices {
  int place, token;
  float gate;
  __device__ __forceinline__ Choices(const MoeRowsArgs &a, int64_t first, int n, int lane, bool want_token) {
    const bool in = lane < n;
    place = in ? a.place[first + lane] : -1;
    token = in && want_token ? a.source[first + lane] : 0;
    gate = in && a.gate ? a.gate[first + lane] : 1.f;
    if (place >= a.t * a.top) place = -1;
    if (token >= a.t) token = -1;
  }
  __device__ __forceinline__ int64_t at(int j) const { return __builtin_amdgcn_readlane(place, j); }   // < 0: none
  __device__ __forceinline__ bool no_token(int j) const { return __builtin_amdgcn_readlane(token, j) < 0; }
  __device__ __forceinline__ float weight(int j) const {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(gate), j));
  }
};

// One wave: token `i`, whole chunks [seg * 64 U, ..) of its rows, U for each lane; the wave of the last ones also
// takes the elements behind them (fewer than a chunk, a lane each). Loads are not guarded: a lane past the last
// chunk, or a choice without a place, reads another place of the array, and what it read is not used (behind a
// branch each load waits for the one before: 54 us instead of 43 on 8192 x 4096 with two choices). KB: rows
// of choices that are requested together.
template <typename T, bool kAl, int U, int KB, bool kGather>
__global__ __launch_bounds__(256) void rows_kernel(MoeRowsArgs a, int64_t segs) {
  using C = Chunk<T, kAl>;
  const int lane = threadIdx.x & 63;
  const int64_t full = a.d / C::P, waves = (int64_t)gridDim.x * 4;
  const int tail = kAl ? 0 : (int)(a.d % C::P);
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < a.t * segs; w += waves) {
    const int64_t i = w / segs, seg = w - i * segs, c0 = seg * 64 * U + lane;
    const bool main = seg * 64 * U < full, last = seg == segs - 1 && lane < tail;
    int64_t at[U];          // first elements of this lane's chunks
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = (c0 + 64 * u < full ? c0 + 64 * u : full - 1) * C::P;
    const int64_t end = full * C::P + lane;        // this lane's element behind the chunks
    const T *x = reinterpret_cast<const T *>(a.x);
    T *out = reinterpret_cast<T *>(a.out);
    C v[kGather ? 1 : KB][U];
    T e[kGather ? 1 : KB];
    if constexpr (kGather) {
      x += i * a.ldx;
      if (main)
#pragma unroll
        for (int u = 0; u < U; ++u) v[0][u].load(x + at[u]);
      if (last) e[0] = x[end];
      auto put = [&](int64_t row, const C *c, T one) {
        if (main)
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c0 + 64 * u < full) c[u].store(out + row * a.d + at[u]);
        if (last) out[row * a.d + end] = one;
      };
      C zero[U];
#pragma unroll
      for (int u = 0; u < U; ++u) zero[u].v = u32x4{0, 0, 0, 0};
      for (int j0 = 0; j0 < a.top; j0 += 64) {
        const int n = a.top - j0 < 64 ? a.top - j0 : 64;
        const Choices ch(a, i * a.top + j0, n, lane, true);
        for (int j = 0; j < n; ++j) {
          if (ch.at(j) >= 0) put(ch.at(j), v[0], e[0]);
          if (ch.no_token(j)) put(i * a.top + j0 + j, zero, (T)0);
        }
      }
    } else {
      float acc[U][C::P], acc_e = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < C::P; ++k) acc[u][k] = 0.f;
      if (a.base) {
        const T *base = reinterpret_cast<const T *>(a.base) + i * a.ldb;
        C b[U];
        if (main) {
#pragma unroll
          for (int u = 0; u < U; ++u) b[u].load(base + at[u]);
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < C::P; ++k) acc[u][k] = b[u].get(k);
        }
        if (last) acc_e = value<T>(base[end]);
      }
      for (int j0 = 0; j0 < a.top; j0 += 64) {
        const int n = a.top - j0 < 64 ? a.top - j0 : 64;
        const Choices ch(a, i * a.top + j0, n, lane, false);
        for (int j = 0; j < n; j += KB) {
          const T *row[KB];
#pragma unroll
          for (int k = 0; k < KB; ++k) {
            const int64_t p = ch.at(j + k < n ? j + k : j);
            row[k] = x + (p >= 0 ? p : 0) * a.d;
          }
          if (main)
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
              for (int u = 0; u < U; ++u) v[k][u].load(row[k] + at[u]);
          if (last)
#pragma unroll
            for (int k = 0; k < KB; ++k) e[k] = row[k][end];
#pragma unroll
          for (int k = 0; k < KB; ++k)
            if (j + k < n && ch.at(j + k) >= 0) {
              const float g = ch.weight(j + k);
              if (main)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                  for (int m = 0; m < C::P; ++m) acc[u][m] += g * v[k][u].get(m);
              if (last) acc_e += g * value<T>(e[k]);
            }
        }
      }
      if (main)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c0 + 64 * u < full) {
            C o;
            o.set(acc[u]);
            o.store(out + i * a.ldo + at[u]);
          }
      if (last) out[i * a.ldo + end] = rounded<T>(acc_e);
    }
  }
}

// One wave: choice j of token i, its rows whole, and the row i * top + j if it has no token. The waves of a
// token's choices are neighbours and find its dY in the caches.
template <typename T, bool kAl>
__global__ __launch_bounds__(256) void rows_bwd_kernel(MoeRowsArgs a) {
  using C = Chunk<T, kAl>;
  constexpr int U = 4;
  const int lane = threadIdx.x & 63;
  const int64_t full = a.d / C::P, waves = (int64_t)gridDim.x * 4;
  const int tail = kAl ? 0 : (int)(a.d % C::P);
  const T *z = reinterpret_cast<const T *>(a.z);
  T *dz = reinterpret_cast<T *>(a.out);
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < a.t * a.top; w += waves) {
    const T *dy = reinterpret_cast<const T *>(a.x) + w / a.top * a.ldx;
    const Choices ch(a, w, 1, lane, true);
    const int64_t p = ch.at(0);
    float dot = 0.f;
    if (p >= 0) {
      const float g = ch.weight(0);
      const T *zp = z + p * a.d;
      T *dzp = dz + p * a.d;
      for (int64_t c = lane; c < full; c += 64 * U) {
        C y[U], v[U];
        int64_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) at[u] = (c + 64 * u < full ? c + 64 * u : full - 1) * C::P;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          y[u].load(dy + at[u]);
          v[u].load(zp + at[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c + 64 * u < full) {
            float f[C::P];
#pragma unroll
            for (int e = 0; e < C::P; ++e) {
              dot += y[u].get(e) * v[u].get(e);
              f[e] = g * y[u].get(e);
            }
            C o;
            o.set(f);
            o.store(dzp + at[u]);
          }
      }
      if (lane < tail) {
        const int64_t e = full * C::P + lane;
        dot += value<T>(dy[e]) * value<T>(zp[e]);
        dzp[e] = rounded<T>(g * value<T>(dy[e]));
      }
      for (int o = 32; o; o >>= 1) dot += __shfl_xor(dot, o);
    }
    if (lane == 0) a.dgate[w] = dot;
    if (ch.no_token(0)) {
      C zero;
      zero.v = u32x4{0, 0, 0, 0};
      for (int64_t c = lane; c < full; c += 64) zero.store(dz + w * a.d + c * C::P);
      if (lane < tail) dz[w * a.d + full * C::P + lane] = (T)0;
    }
  }
}

template <typename T, bool kAl, int U, bool kGather>
void launch_rows_wide(const MoeRowsArgs &a, hipStream_t st) {
  const int64_t full = a.d / Chunk<T, kAl>::P, segs = full ? (full + 64 * U - 1) / (64 * U) : 1;
  int64_t blocks = (a.t * segs + 3) / 4;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  const dim3 g((unsigned)blocks), b(256);
  if constexpr (kGather) {
    rows_kernel<T, kAl, U, 1, true><<<g, b, 0, st>>>(a, segs);
  } else {
    if (a.top == 1) rows_kernel<T, kAl, U, 1, false><<<g, b, 0, st>>>(a, segs);
    else if (a.top == 2) rows_kernel<T, kAl, U, 2, false><<<g, b, 0, st>>>(a, segs);
    else rows_kernel<T, kAl, U, 4, false><<<g, b, 0, st>>>(a, segs);
  }
}

template <typename T, bool kAl, bool kGather>
hipError_t launch_rows_as(const MoeRowsArgs &a, hipStream_t st) {
  const int64_t full = a.d / Chunk<T, kAl>::P;
  // four chunks a lane once that still gives every CU 16 waves
  if (a.t * ((full + 255) / 256) >= 4096) launch_rows_wide<T, kAl, 4, kGather>(a, st);
  else launch_rows_wide<T, kAl, 1, kGather>(a, st);
  return hipGetLastError();
}

bool vec_rows(const MoeRowsArgs &a, size_t esz) {
  uintptr_t all = (uintptr_t)a.x | (uintptr_t)a.out | (uintptr_t)a.z | (uintptr_t)a.base;
  all |= (uintptr_t)((a.d | a.ldx | a.ldo | a.ldb) * (int64_t)esz);
  return (all & 15) == 0;
}

}  // namespace

hipError_t launch_gather(const MoeRowsArgs &a, bool f32, hipStream_t st) {
  if (vec_rows(a, f32 ? 4 : 2))
    return f32 ? launch_rows_as<float, true, true>(a, st) : launch_rows_as<uint16_t, true, true>(a, st);
  return f32 ? launch_rows_as<float, false, true>(a, st) : launch_rows_as<uint16_t, false, true>(a, st);
}

hipError_t launch_combine(const MoeRowsArgs &a, bool f32, hipStream_t st) {
  if (vec_rows(a, f32 ? 4 : 2))
    return f32 ? launch_rows_as<float, true, false>(a, st) : launch_rows_as<uint16_t, true, false>(a, st);
  return f32 ? launch_rows_as<float, false, false>(a, st) : launch_rows_as<uint16_t, false, false>(a, st);
}

hipError_t launch_combine_bwd(const MoeRowsArgs &a, bool f32, hipStream_t st) {
  int64_t blocks = (a.t * a.top + 3) / 4;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  const dim3 g((unsigned)blocks), b(256);
  if (vec_rows(a, f32 ? 4 : 2)) {
    if (f32) rows_bwd_kernel<float, true><<<g, b, 0, st>>>(a);
    else rows_bwd_kernel<uint16_t, true><<<g, b, 0, st>>>(a);
  } else {
    if (f32) rows_bwd_kernel<float, false><<<g, b, 0, st>>>(a);
    else rows_bwd_kernel<uint16_t, false><<<g, b, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace nf4q
