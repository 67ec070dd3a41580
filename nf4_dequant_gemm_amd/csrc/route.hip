// Choice of experts for the grouped layer, and its gradient (gfx950).
//
// For the logits x of one token over E experts, p = softmax(x) and lse = log sum exp(x):
//
//   chosen   the `top` largest x, ties to the lower index; -inf is never chosen
//   gate_k   p of the k-th choice, or the softmax over the chosen logits alone (renormalised)
//   place    the row of a choice when all of them are ordered by expert, then by token
//   balance  E sum_e (counts_e / N) mean_p_e,   z = mean lse^2
//
// over the n routed tokens and their N choices; a token with keep 0 or without a logit above -inf is not
// routed. The counts are constants of the gradient:
//
//   dx_e = p_e (c_e - sum p c) + (2 dz / n) lse p_e + the gates' part,   c_e = dbalance E counts_e / (N n)
//   gates as they are:  c_e also holds dgate_k of the chosen;   renormalised:  g_k (dg_k - sum g dg).
//
// What bounds it is latency, not the few megabytes of logits. 16 lanes take a token, expert l + 16 j in
// register j of lane l, so that a choice is a scan of the registers, a maximum over the lanes in four
// cross-lane moves, and a second such step for the lowest index. Logits are compared as unsigned integers
// in the same order (NaN above everything, so that a row with NaN still chooses `top` different experts),
// 0 means not to be chosen. Places need the counts of the blocks before, hence two launches (one for as
// many tokens as a workgroup takes at once); a block's places come from one bit mask of 64 tokens for each
// expert: the rank of a choice is the number of lower bits, in any order of the atomics. The sums of p go
// from registers through fixed orders, so that all results are the same on every call.
//
// Measured: one token, 128 experts, top 8: 6.0 us; 16384 tokens of 128 float32 logits, top 8: choices 10.4 us (of
// which the vector instructions of 16 waves a CU are about half), places 8.6 us, gradient 8.9 us (16 MB).
#include "common.h"
#include "launch.h"

namespace nf4q {
namespace {

constexpr int kE = kMaxExperts;
static_assert(kE == 256 && kRouteMaxTop == 16, "16 lanes of 16 experts, a lane for each choice");

template <typename XT>
__device__ __forceinline__ float to_f32(XT v);
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }

// Value of v `n` lanes further within each 16 (DPP row rotation); over 8, 4, 2 and 1 every lane meets all.
template <int n>
__device__ __forceinline__ uint32_t turn(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + n, 0xF, 0xF, true);
}
template <typename F>
__device__ __forceinline__ uint32_t over16(uint32_t v, F f) {
  v = f(v, turn<8>(v));
  v = f(v, turn<4>(v));
  v = f(v, turn<2>(v));
  return f(v, turn<1>(v));
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  return over16(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t min16(uint32_t v) {
  return over16(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
__device__ __forceinline__ float sum16(float v) {
  return __uint_as_float(over16(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// The logits of a lane's experts l + 16 j, all requested at once (the last expert's in the place of one past it; a
// branch around each load made eight trips to memory of them).
template <typename XT, int NV>
__device__ __forceinline__ void load_row(const XT *x, int l, int E, float *v) {
  XT raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) raw[j] = x[l + 16 * j < E ? l + 16 * j : E - 1];
#pragma unroll
  for (int j = 0; j < NV; ++j) v[j] = to_f32<XT>(raw[j]);
}

// A logit as an integer of the same order: 0 for -inf (never chosen), the largest for NaN, +0 for -0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t k = b ^ (uint32_t)((int32_t)b >> 31 | (int32_t)0x80000000);
  return x != x ? 0xFFFFFFFFu : x == -INFINITY ? 0u : k;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

struct Shared {
  float psum[16][kE];        // by wave
  float z[16], red[4];
  int n[16];
  int hist[kE], base[kE], total;
  unsigned long long mask[kE];
};

// base[e] = the first row of expert e, from the counts [E]; returns the number of rows. Whole workgroup.
__device__ __forceinline__ int first_rows(const int *counts, int E, int *base, int *total) {
  const int tid = threadIdx.x;
  if (tid < 64) {
    int c[4], s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 4 * tid + i < E ? counts[4 * tid + i] : 0;
      s += c[i];
    }
    int up = s;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(up, o);
      if (tid >= o) up += v;
    }
    int at = up - s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * tid + i < E) base[4 * tid + i] = at;
      at += c[i];
    }
    if (tid == 63) *total = up;
  }
  __syncthreads();
  return *total;
}

// Places and sources of the tokens [lo, hi), with base[e] the first row of expert e that is theirs. A thread takes
// one choice of up to 64 tokens (64 * kRouteMaxTop <= blockDim.x); `e` is its expert among the first of them, whose
// mask bits are set.
__device__ __forceinline__ void place_rows(const RouteArgs &a, int64_t lo, int64_t hi, int e, int *base,
                                           unsigned long long *mask) {
  const int tid = threadIdx.x, top = a.top, row = tid / top;
  for (int64_t c0 = lo;;) {
    if (row < 64 && c0 + row < hi) {
      int at = -1;
      if (e >= 0) {
        at = base[e] + __popcll(mask[e] & ((1ull << row) - 1));
        a.source[at] = (int)(c0 + row);
      }
      a.place[c0 * top + tid] = at;
    }
    c0 += 64;
    if (c0 >= hi) return;
    __syncthreads();
    if (tid < a.E) {
      base[tid] += __popcll(mask[tid]);
      mask[tid] = 0;
    }
    __syncthreads();
    e = row < 64 && c0 + row < hi ? a.idx[c0 * top + tid] : -1;
    if (e >= 0) atomicOr(&mask[e], 1ull << row);
    __syncthreads();
  }
}

// Counts, sizes, mean probabilities and losses from the totals. Whole workgroup, E <= its threads;
// red: 2 x 16 floats of LDS.
__device__ __forceinline__ void finish(const RouteArgs &a, int count, float psum, float z, int n, int rows, float *red) {
  const int tid = threadIdx.x;
  float part = 0.f;
  if (tid < a.E) {
    a.counts[tid] = count;
    const float mean = n ? psum / (float)n : 0.f;
    a.mean_p[tid] = mean;
    part = rows ? mean * ((float)count / (float)rows) : 0.f;
  }
  for (int o = 32; o; o >>= 1) part += __shfl_xor(part, o);
  if (tid < kE && (tid & 63) == 0) red[tid >> 6] = part;
  __syncthreads();
  if (tid == 0) {
    a.losses[0] = (float)a.E * (red[0] + red[1] + red[2] + red[3]);
    a.losses[1] = n ? z / (float)n : 0.f;
    a.sizes[0] = n;
    a.sizes[1] = rows;
  }
}

// Block b chooses for its a.rows tokens. A single block (at most 64 tokens, one for each group of 16 lanes) goes on
// to the places and totals; more leave their counts [Ep], sums of p [Ep], of lse^2 and numbers of tokens for
// route_place_kernel.
template <typename XT, int NV>
__global__ __launch_bounds__(1024) void route_choose_kernel(RouteArgs a) {
  __shared__ Shared s;
  const int tid = threadIdx.x, l = tid & 15, groups = blockDim.x / 16, top = a.top, E = a.E;
  const bool one = gridDim.x == 1;
  const int64_t lo = (int64_t)blockIdx.x * a.rows;
  const int64_t hi = lo + a.rows < a.t ? lo + a.rows : a.t;
  for (int e = tid; e < kE; e += blockDim.x) {
    s.hist[e] = 0;
    s.mask[e] = 0;
  }
  __syncthreads();

  int my_e = -1;
  float psum[NV], zsum = 0.f;
  int nsum = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) psum[j] = 0.f;
  for (int64_t row = lo + tid / 16; row < hi; row += groups) {   // whole groups of 16 lanes
    const XT *x = reinterpret_cast<const XT *>(a.x) + row * a.ld;
    const bool keep = !a.keep || a.keep[row];
    uint32_t key[NV];
    float v[NV];
    load_row<XT, NV>(x, l, E, v);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      key[j] = keep && l + 16 * j < E ? key_of(v[j]) : 0u;
      v[j] = key[j] ? v[j] : -INFINITY;
    }
    // lane k gets choice k
    my_e = -1;
    uint32_t my_key = 0, first = 0;
    for (int k = 0; k < top; ++k) {
      uint32_t best = 0;
      int bj = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (key[j] > best) {
          best = key[j];
          bj = j;
        }
      const uint32_t m = max16(best);
      const int e = (int)min16(best == m ? (uint32_t)(l + 16 * bj) : 0xFFFFu);
      if (k == 0) first = m;
      if (m == 0) break;     // nothing left to choose, the same in all 16 lanes
      if (l == k) {
        my_e = e;
        my_key = m;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (e == l + 16 * j) key[j] = 0;
    }
    float gate = 0.f;
    if (first) {
      const float mx = of_key(first);
      float ev[NV], sum = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        ev[j] = expf(v[j] - mx);
        sum += ev[j];
      }
      sum = sum16(sum);
      const float mine = my_e >= 0 ? expf(of_key(my_key) - mx) : 0.f;
      gate = mine / (a.renorm ? sum16(mine) : sum);
      const float inv = 1.f / sum;
#pragma unroll
      for (int j = 0; j < NV; ++j) psum[j] += ev[j] * inv;
      const float lse = mx + logf(sum);
      zsum += lse * lse;
      nsum += 1;
    }
    if (l < top) {
      a.idx[row * top + l] = my_e;
      a.gate[row * top + l] = gate;
      if (my_e >= 0) {
        if (one) atomicOr(&s.mask[my_e], 1ull << row);
        else atomicAdd(&s.hist[my_e], 1);
      }
    }
  }

  // sums of the wave's four groups, then of the waves, in a fixed order
  const int lane = tid & 63, wave = tid >> 6, waves = blockDim.x / 64;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    psum[j] += __shfl_xor(psum[j], 16);
    psum[j] += __shfl_xor(psum[j], 32);
    if (lane < 16) s.psum[wave][l + 16 * j] = psum[j];
  }
  zsum += __shfl_xor(zsum, 16);
  zsum += __shfl_xor(zsum, 32);
  nsum += __shfl_xor(nsum, 16);
  nsum += __shfl_xor(nsum, 32);
  if (lane == 0) {
    s.z[wave] = zsum;
    s.n[wave] = nsum;
  }
  __syncthreads();
  float z = 0.f, p = 0.f;
  int n = 0;
  for (int w = 0; w < waves; ++w) {
    z += s.z[w];
    n += s.n[w];
    if (tid < 16 * NV) p += s.psum[w][tid];
  }
  if (!one) {
    const int64_t b = blockIdx.x;
    if (tid < a.Ep) {
      a.cnt[b * a.Ep + tid] = s.hist[tid];
      a.psum[b * a.Ep + tid] = p;
    }
    if (tid == 0) {
      a.zsum[b] = z;
      a.nsum[b] = n;
    }
    return;
  }
  const int count = tid < kE ? __popcll(s.mask[tid]) : 0;
  if (tid < kE) s.hist[tid] = count;
  __syncthreads();
  const int rows = first_rows(s.hist, E, s.base, &s.total);
  const int64_t row = tid / 16;
  if (row < hi && l < top) {
    int at = -1;
    if (my_e >= 0) {
      at = s.base[my_e] + __popcll(s.mask[my_e] & ((1ull << row) - 1));
      a.source[at] = (int)row;
    }
    a.place[row * top + l] = at;
  }
  for (int64_t i = rows + tid; i < a.t * top; i += blockDim.x) a.source[i] = -1;
  finish(a, count, p, z, n, rows, s.red);
}

// Block b < a.blocks: the places of its tokens; the last block: counts, mean probabilities and losses. Two blocks
// have to fit on a CU (64 registers): with 256 blocks of tokens the last one otherwise starts when the first ends.
__global__ __launch_bounds__(1024, 8) void route_place_kernel(RouteArgs a) {
  constexpr int kSlices = 32;
  __shared__ __align__(16) int s_tot[4096], s_bef[4096];     // [slices][Ep]: four for each thread
  __shared__ int s_base[kE], s_cnt[kE], s_total;
  __shared__ unsigned long long s_mask[kE];
  __shared__ float s_red[4];
  const int tid = threadIdx.x, b = blockIdx.x, quads = a.Ep / 4;
  const bool last = b == a.blocks;
  const int64_t lo = (int64_t)b * a.rows, hi = lo + a.rows < a.t ? lo + a.rows : a.t;
  const int row = tid / a.top;
  const int e = row < 64 && lo + row < hi ? a.idx[lo * a.top + tid] : -1;      // of the first 64 tokens
  if (tid < kE) s_mask[tid] = 0;
  int slices = (int)blockDim.x / quads;
  slices = slices < kSlices ? slices : kSlices;
  const int sl = tid / quads, q = tid % quads;
  if (sl < slices) {
    int4 tot = make_int4(0, 0, 0, 0), bef = tot;
#pragma unroll 8
    for (int i = sl; i < a.blocks; i += slices) {
      const int4 c = *reinterpret_cast<const int4 *>(a.cnt + (int64_t)i * a.Ep + 4 * q);
      const int in = i < b ? -1 : 0;
      tot.x += c.x, tot.y += c.y, tot.z += c.z, tot.w += c.w;
      bef.x += c.x & in, bef.y += c.y & in, bef.z += c.z & in, bef.w += c.w & in;
    }
    *reinterpret_cast<int4 *>(&s_tot[sl * a.Ep + 4 * q]) = tot;
    *reinterpret_cast<int4 *>(&s_bef[sl * a.Ep + 4 * q]) = bef;
  }
  __syncthreads();
  if (e >= 0) atomicOr(&s_mask[e], 1ull << row);
  int tot = 0, bef = 0;
  if (tid < a.Ep) {
    for (int i = 0; i < slices; ++i) {
      tot += s_tot[i * a.Ep + tid];
      bef += s_bef[i * a.Ep + tid];
    }
    s_cnt[tid] = tot;
  }
  __syncthreads();
  const int rows = first_rows(s_cnt, a.E, s_base, &s_total);
  if (!last) {
    if (tid < a.E) s_base[tid] += bef;
    for (int64_t i = rows + (int64_t)b * blockDim.x + tid; i < a.t * a.top; i += (int64_t)a.blocks * blockDim.x)
      a.source[i] = -1;
    __syncthreads();
    place_rows(a, lo, hi, e, s_base, s_mask);
    return;
  }
  // sums of p: slices of blocks as above, in the memory of s_bef
  float *sp = reinterpret_cast<float *>(s_bef);
  if (sl < slices) {
    f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int i = sl; i < a.blocks; i += slices) p += *reinterpret_cast<const f32x4 *>(a.psum + (int64_t)i * a.Ep + 4 * q);
    *reinterpret_cast<f32x4 *>(&sp[sl * a.Ep + 4 * q]) = p;
  }
  float z = tid < a.blocks ? a.zsum[tid] : 0.f;     // at most kRouteMaxBlocks, within four waves
  int n = tid < a.blocks ? a.nsum[tid] : 0;
  for (int o = 32; o; o >>= 1) {
    z += __shfl_xor(z, o);
    n += __shfl_xor(n, o);
  }
  __shared__ float s_z[16];
  __shared__ int s_n[16];
  if ((tid & 63) == 0) {
    s_z[tid >> 6] = z;
    s_n[tid >> 6] = n;
  }
  __syncthreads();
  float p = 0.f;
  if (tid < a.E)
    for (int i = 0; i < slices; ++i) p += sp[i * a.Ep + tid];
  static_assert(kRouteMaxBlocks == 256, "four waves");
  finish(a, tot, p, s_z[0] + s_z[1] + s_z[2] + s_z[3], s_n[0] + s_n[1] + s_n[2] + s_n[3], rows, s_red);
}

template <typename XT, int NV>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs a) {
  const int tid = threadIdx.x, l = tid & 15, E = a.E, top = a.top;
  // requested here, used behind the first row's requests: one trip to memory
  const int64_t n = a.sizes[0], rows = a.sizes[1];
  int64_t count[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) count[j] = a.counts[l + 16 * j < E ? l + 16 * j : E - 1];
  const float db = a.dlosses ? a.dlosses[0] : 0.f, dz = a.dlosses ? a.dlosses[1] : 0.f;
  for (int64_t row = (int64_t)blockIdx.x * 16 + tid / 16; row < a.t; row += (int64_t)gridDim.x * 16) {
    const XT *x = reinterpret_cast<const XT *>(a.x) + row * a.ld;
    XT *dx = reinterpret_cast<XT *>(a.dx) + row * a.ldd;
    int e = l < top ? a.idx[row * top + l] : -1;
    float dg = a.dgate && l < top ? a.dgate[row * top + l] : 0.f;
    float v[NV], d[NV];
    load_row<XT, NV>(x, l, E, v);
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = l + 16 * j < E ? v[j] : -INFINITY;
    if (e >= E) e = -1;
    if (max16((uint32_t)(e + 1)) == 0) {       // not routed
#pragma unroll
      for (int j = 0; j < NV; ++j) d[j] = 0.f;
    } else {
      const float xe = e >= 0 ? to_f32<XT>(x[e]) : 0.f;
      if (e < 0) dg = 0.f;
      float mx = -INFINITY, sum = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) mx = fmaxf(mx, v[j]);
      mx = __uint_as_float(over16(__float_as_uint(mx), [](uint32_t p, uint32_t q) {
        return __float_as_uint(fmaxf(__uint_as_float(p), __uint_as_float(q)));
      }));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        v[j] = expf(v[j] - mx);
        sum += v[j];
      }
      sum = sum16(sum);
      const float inv = 1.f / sum;
      const float pe = e >= 0 ? expf(xe - mx) : 0.f;
      const float g = pe / (a.renorm ? sum16(pe) : sum);
      float w = g * dg;
      const float mean = sum16(w);
      if (a.renorm) w -= g * mean;
      const float k = db * (float)E / (float)n / (float)rows, zc = 2.f * dz / (float)n;
      float c[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        c[j] = k * (float)count[j];
        v[j] *= inv;
        dot += v[j] * c[j];
      }
      dot = sum16(dot);
      if (!a.renorm) dot += mean;
      const float zl = zc * (mx + logf(sum));
#pragma unroll
      for (int j = 0; j < NV; ++j) d[j] = v[j] * (c[j] - dot + zl);
      for (int k = 0; k < top; ++k) {
        const int ek = __shfl(e, k, 16);
        const float wk = __shfl(w, k, 16);
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (ek == l + 16 * j) d[j] += wk;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (l + 16 * j < E) {
        if constexpr (sizeof(XT) == 2)
          dx[l + 16 * j] = (uint16_t)(pack_bf16x2(d[j], 0.f) & 0xFFFFu);
        else
          dx[l + 16 * j] = d[j];
      }
  }
}

}  // namespace

RoutePlan route_plan(int64_t t, int E) {
  RoutePlan p;
  p.Ep = (E + 15) / 16 * 16;
  // at most 64 tokens: one workgroup of 16 lanes a token; otherwise 16 tokens a workgroup, and more of
  // them (up to 64 at once, in up to 1024 threads) where that would be over 256 workgroups
  p.rows = t <= 64 ? (t <= 16 ? 16 : 64) : 16 * ((t + 16 * kRouteMaxBlocks - 1) / (16 * kRouteMaxBlocks));
  p.blocks = t > 0 ? (int)((t + p.rows - 1) / p.rows) : 1;      // without tokens the totals are still written
  p.threads = p.rows >= 64 ? 1024 : 16 * (int)p.rows;
  p.bytes = p.blocks > 1 ? (size_t)p.blocks * (8 * p.Ep + 8) : 0;
  return p;
}

#define ROUTE_FOR(kernel, grid, threads, st)                                            \
  do {                                                                                  \
    const int nv = (a.E + 15) / 16;                                                     \
    if (nv <= 1) { ROUTE_TYPE(kernel, 1, grid, threads, st); }                          \
    else if (nv <= 2) { ROUTE_TYPE(kernel, 2, grid, threads, st); }                     \
    else if (nv <= 4) { ROUTE_TYPE(kernel, 4, grid, threads, st); }                     \
    else if (nv <= 8) { ROUTE_TYPE(kernel, 8, grid, threads, st); }                     \
    else { ROUTE_TYPE(kernel, 16, grid, threads, st); }                                 \
  } while (0)
#define ROUTE_TYPE(kernel, nv, grid, threads, st)                                       \
  if (f32) kernel<float, nv><<<dim3(grid), dim3(threads), 0, st>>>(a);                  \
  else kernel<uint16_t, nv><<<dim3(grid), dim3(threads), 0, st>>>(a)

hipError_t launch_route(RouteArgs a, bool f32, void *ws, hipStream_t st) {
  const RoutePlan p = route_plan(a.t, a.E);
  if (a.E < 1 || a.E > kE || a.top < 1 || a.top > kRouteMaxTop || a.top > a.E || p.blocks > kRouteMaxBlocks)
    return hipErrorInvalidValue;
  a.rows = p.rows;
  a.blocks = p.blocks;
  a.Ep = p.Ep;
  a.cnt = (int *)ws;
  a.psum = (float *)ws + (int64_t)p.blocks * p.Ep;
  a.zsum = a.psum + (int64_t)p.blocks * p.Ep;
  a.nsum = (int *)(a.zsum + p.blocks);
  ROUTE_FOR(route_choose_kernel, (unsigned)p.blocks, (unsigned)p.threads, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.blocks == 1) return e;
  route_place_kernel<<<dim3((unsigned)p.blocks + 1), dim3(1024), 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdArgs &a, bool f32, hipStream_t st) {
  if (a.E < 1 || a.E > kE || a.top < 1 || a.top > kRouteMaxTop) return hipErrorInvalidValue;
  int64_t blocks = (a.t + 15) / 16;
  if (blocks > 4096) blocks = 4096;
  ROUTE_FOR(route_bwd_kernel, (unsigned)blocks, 256, st);
  return hipGetLastError();
}

}  // namespace nf4q
