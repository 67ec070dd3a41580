// Norm of every query and key head with the position rotation in the same pass, and its backward
// (gfx950): what follows the q and k projections.
//
//   xh = x / sqrt(mean(x^2) + eps),   n = xh * (w + offset),   y = R(pos) n
//
// over one head x[0 .. d): R turns the pairs of the first `rot` elements by the token's angles,
// (a, b) -> (a cos - b sin, a sin + b cos), pairs (i, i + rot/2) or, interleaved, (2i, 2i + 1); the
// elements past `rot` pass through. Backward, from g = dL/dy:
//
//   gn = R(pos)^T g,   dw = sum gn * xh,   gh = gn * (w + offset),
//   dx = (gh - xh mean(gh * xh)) / sqrt(mean(x^2) + eps)
//
// with mean(x^2) formed again from x (no statistics kept). Sums are in float32; y and dx are rounded
// once, to the type of x.
//
// Work split. Both directions read and write each element once: they are memory bound. A head is
// cut into units of two chunks of kVec elements, the two a rotation pairs up (i and i + rot/2; for
// interleaved pairs two neighbouring chunks), so that the rotation needs no exchange between
// lanes: a lane holds both members of each of its pairs. A head's units take the first lanes of a
// power of two of lanes, whose float sums meet by lane exchanges; kVec is the largest power of two
// up to 16 bytes that divides rot/2, d - rot, the strides and the addresses. Threads keep their unit and walk over
// (token, head) items, so the weight stays in registers; q and k items go to separate workgroups,
// and dw is summed in registers over a thread's items, over the workgroup in LDS and over the
// workgroups by a second launch, in an order that the sizes alone fix.
#include "common.h"
#include "launch.h"

namespace nf4q {
namespace {

constexpr int kThreads = 256;

template <typename XT>
struct Elem;
template <>
struct Elem<uint16_t> {
  static __device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ uint16_t from_f32(float v) {
    return (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
  }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float to_f32(float v) { return v; }
  static __device__ __forceinline__ float from_f32(float v) { return v; }
};

template <typename XT, int kVec>
struct alignas(sizeof(XT) * kVec) Chunk {
  XT v[kVec];
};

template <typename XT, int kVec>
__device__ __forceinline__ void load_chunk(const XT *p, float out[kVec]) {
  const Chunk<XT, kVec> c = *reinterpret_cast<const Chunk<XT, kVec> *>(p);
#pragma unroll
  for (int i = 0; i < kVec; ++i) out[i] = Elem<XT>::to_f32(c.v[i]);
}
template <typename XT, int kVec>
__device__ __forceinline__ void store_chunk(XT *p, const float in[kVec]) {
  Chunk<XT, kVec> c;
#pragma unroll
  for (int i = 0; i < kVec; ++i) c.v[i] = Elem<XT>::from_f32(in[i]);
  // Streamed out, since it is not read again here: forward and backward of 8192 tokens of 40 heads of 128 take
  // 98.5 us, 103 without; the forward alone 35.6 and 32.5 in bf16 (the outputs then stay in the last cache),
  // 61.3 and 63.3 in float32.
  if constexpr (sizeof(c) == 16)
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, c), reinterpret_cast<u32x4 *>(p));
  else
    *reinterpret_cast<Chunk<XT, kVec> *>(p) = c;
}

// Sum over the `lph` (a power of two) neighbouring lanes that hold a head.
__device__ __forceinline__ float head_sum(float v, int lph) {
  for (int o = 1; o < lph; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// kVec elements a chunk, kUnits units a lane (more than one only for heads of more than 64 units).
template <typename XT, int kVec, int kUnits, bool kInter, bool kBwd>
__global__ __launch_bounds__(kThreads) void head_norm_kernel(HeadArgs a) {
  extern __shared__ float sdw[];   // backward: [waves][d]
  const bool is_k = (int)blockIdx.x >= a.blocks_q;
  const HeadSide &h = is_k ? a.k : a.q;
  const int nblocks = is_k ? (int)gridDim.x - a.blocks_q : a.blocks_q;
  const int block = is_k ? (int)blockIdx.x - a.blocks_q : (int)blockIdx.x;
  const int lph = a.lanes, d = a.d, rot = a.rot, half = rot / 2;
  const int unit0 = threadIdx.x & (lph - 1);
  const int per_block = kThreads / lph;            // heads a workgroup holds at once
  const int rot_units = half / kVec;
  const float inv_d = 1.f / (float)d;
  const int64_t items = a.m * h.heads;

  // this lane's units: places of the two chunks (-1: none) and the weight there
  int pa[kUnits], pb[kUnits];
  float wa[kUnits][kVec], wb[kUnits][kVec];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int unit = unit0 + u * lph;
    if (unit < rot_units) {
      pa[u] = kInter ? 2 * unit * kVec : unit * kVec;
      pb[u] = kInter ? pa[u] + kVec : half + unit * kVec;
    } else {
      pa[u] = rot + 2 * (unit - rot_units) * kVec;
      pb[u] = pa[u] + kVec;
      if (pa[u] >= d) pa[u] = -1;
      if (pb[u] >= d) pb[u] = -1;
    }
    auto weight = [&](int p, float *w) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) w[i] = 0.f;
      if (p < 0) return;
      if (a.w_f32)
        load_chunk<float, kVec>(reinterpret_cast<const float *>(h.w) + p, w);
      else
        load_chunk<uint16_t, kVec>(reinterpret_cast<const uint16_t *>(h.w) + p, w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) w[i] += a.w_offset;
    };
    weight(pa[u], wa[u]);
    weight(pb[u], wb[u]);
  }
  float da[kUnits][kVec], db[kUnits][kVec];        // backward: this thread's part of dw
  if constexpr (kBwd) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < kVec; ++i) da[u][i] = db[u][i] = 0.f;
  }

  // Rotation of one unit by (cos, sin) or, backward, by its transpose (sin of the other sign).
  auto turn = [&](float *x, float *y, const float *c, const float *s, float sign) {
    if constexpr (kInter && kVec > 1) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {             // pair i: elements 2 i, 2 i + 1 of [x | y]
        float *p = i < kVec / 2 ? x + 2 * i : y + 2 * i - kVec;
        const float u = p[0] * c[i] - sign * p[1] * s[i], v = p[1] * c[i] + sign * p[0] * s[i];
        p[0] = u;
        p[1] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float u = x[i] * c[i] - sign * y[i] * s[i], v = y[i] * c[i] + sign * x[i] * s[i];
        x[i] = u;
        y[i] = v;
      }
    }
  };

  const uint32_t stride = (uint32_t)nblocks * per_block;   // items fit 31 bits (checked at launch)
#pragma unroll 1
  for (uint32_t it = (uint32_t)block * per_block + threadIdx.x / lph; it < (uint32_t)items; it += stride) {
    const uint32_t tok = it / (uint32_t)h.heads, head = it - tok * (uint32_t)h.heads;
    int64_t pos = 0;
    if (rot > 0)
      pos = a.pos64 ? reinterpret_cast<const int64_t *>(a.pos)[tok]
                    : (int64_t) reinterpret_cast<const int32_t *>(a.pos)[tok];
    const XT *x = reinterpret_cast<const XT *>(h.x) + tok * h.x_ts + head * h.x_hs;
    float xa[kUnits][kVec], xb[kUnits][kVec], ga[kUnits][kVec], gb[kUnits][kVec];
    float cs[kUnits][kVec], sn[kUnits][kVec];
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) xa[u][i] = xb[u][i] = 0.f;
      if (pa[u] >= 0) load_chunk<XT, kVec>(x + pa[u], xa[u]);
      if (pb[u] >= 0) load_chunk<XT, kVec>(x + pb[u], xb[u]);
      if constexpr (kBwd) {
        const XT *g = reinterpret_cast<const XT *>(h.g) + tok * h.g_ts + head * h.g_hs;
#pragma unroll
        for (int i = 0; i < kVec; ++i) ga[u][i] = gb[u][i] = 0.f;
        if (pa[u] >= 0) load_chunk<XT, kVec>(g + pa[u], ga[u]);
        if (pb[u] >= 0) load_chunk<XT, kVec>(g + pb[u], gb[u]);
      }
    }
    // a position outside the table reads nothing there: the token's outputs are NaN
    const bool placed = rot == 0 || (pos >= 0 && pos < a.places);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = unit0 + u * lph;
      if (unit < rot_units && placed) {
        load_chunk<float, kVec>(a.cos + pos * half + unit * kVec, cs[u]);
        load_chunk<float, kVec>(a.sin + pos * half + unit * kVec, sn[u]);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          cs[u][i] = 1.f;
          sn[u][i] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) ss += xa[u][i] * xa[u][i] + xb[u][i] * xb[u][i];
    }
    ss = head_sum(ss, lph);
    float inv = rsqrtf(ss * inv_d + a.eps);
    if (!placed) inv = __builtin_nanf("");
    XT *y = reinterpret_cast<XT *>(h.y) + tok * h.y_ts + head * h.y_hs;
    if constexpr (!kBwd) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          xa[u][i] *= inv * wa[u][i];
          xb[u][i] *= inv * wb[u][i];
        }
        if (unit0 + u * lph < rot_units) turn(xa[u], xb[u], cs[u], sn[u], 1.f);
        if (pa[u] >= 0) store_chunk<XT, kVec>(y + pa[u], xa[u]);
        if (pb[u] >= 0) store_chunk<XT, kVec>(y + pb[u], xb[u]);
      }
    } else {
      float dot = 0.f;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        if (unit0 + u * lph < rot_units) turn(ga[u], gb[u], cs[u], sn[u], -1.f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          xa[u][i] *= inv;
          xb[u][i] *= inv;
          da[u][i] += ga[u][i] * xa[u][i];
          db[u][i] += gb[u][i] * xb[u][i];
          ga[u][i] *= wa[u][i];
          gb[u][i] *= wb[u][i];
          dot += ga[u][i] * xa[u][i] + gb[u][i] * xb[u][i];
        }
      }
      dot = head_sum(dot, lph) * inv_d;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          ga[u][i] = inv * (ga[u][i] - xa[u][i] * dot);
          gb[u][i] = inv * (gb[u][i] - xb[u][i] * dot);
        }
        if (pa[u] >= 0) store_chunk<XT, kVec>(y + pa[u], ga[u]);
        if (pb[u] >= 0) store_chunk<XT, kVec>(y + pb[u], gb[u]);
      }
    }
  }

  if constexpr (kBwd) {
    // dw of the workgroup: the lanes of a wave with the same unit, then the waves in order
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        for (int o = lph; o < 64; o <<= 1) {
          da[u][i] += __shfl_xor(da[u][i], o);
          db[u][i] += __shfl_xor(db[u][i], o);
        }
        if ((int)(threadIdx.x & 63) < lph) {
          if (pa[u] >= 0) sdw[wave * d + pa[u] + i] = da[u][i];
          if (pb[u] >= 0) sdw[wave * d + pb[u] + i] = db[u][i];
        }
      }
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) s += sdw[w * d + c];
      a.part[(int64_t)blockIdx.x * d + c] = s;
    }
  }
}

// dw from the workgroups' parts [blocks][d]: workgroup (c, side) adds 32 columns, 32 threads a
// column over every 32nd part, then in LDS in order.
constexpr int kFinCols = 32, kFinRows = 32;
__global__ __launch_bounds__(kFinCols *kFinRows) void head_norm_dw_kernel(
    const float *__restrict__ part, int d, int blocks_q, int blocks_k, float *__restrict__ dwq,
    float *__restrict__ dwk) {
  __shared__ float red[kFinRows][kFinCols + 1];
  const int col = threadIdx.x % kFinCols, row = threadIdx.x / kFinCols;
  const int c = blockIdx.x * kFinCols + col;
  const bool is_k = blockIdx.y != 0;
  const int lo = is_k ? blocks_q : 0, n = is_k ? blocks_k : blocks_q;
  float s = 0.f;
  if (c < d) {
    const float *p = part + (int64_t)lo * d + c;
    int b = row;
    for (; b + 7 * kFinRows < n; b += 8 * kFinRows) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[(int64_t)(b + j * kFinRows) * d];
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
    for (; b < n; b += kFinRows) s += p[(int64_t)b * d];
  }
  red[row][col] = s;
  __syncthreads();
  if (row == 0 && c < d) {
    s = red[0][col];
    for (int r = 1; r < kFinRows; ++r) s += red[r][col];
    float *out = is_k ? dwk : dwq;
    if (out) out[c] = s;
  }
}

template <typename XT, int kVec, int kUnits>
hipError_t launch_vec(const HeadArgs &a, bool inter, bool bwd, int blocks, hipStream_t st) {
  const dim3 grid((unsigned)blocks), block(kThreads);
  const size_t lds = bwd ? (size_t)(kThreads / 64) * a.d * sizeof(float) : 0;
  if (bwd) {
    if (inter)
      head_norm_kernel<XT, kVec, kUnits, true, true><<<grid, block, lds, st>>>(a);
    else
      head_norm_kernel<XT, kVec, kUnits, false, true><<<grid, block, lds, st>>>(a);
  } else {
    if (inter)
      head_norm_kernel<XT, kVec, kUnits, true, false><<<grid, block, lds, st>>>(a);
    else
      head_norm_kernel<XT, kVec, kUnits, false, false><<<grid, block, lds, st>>>(a);
  }
  return hipGetLastError();
}

// The chunk: the largest power of two up to 16 bytes that divides rot/2, the pass-through part, every
// stride and every address.
int chunk_of(const HeadArgs &a, bool f32, bool bwd) {
  const int esz = f32 ? 4 : 2;
  uint64_t all = (uint64_t)(a.rot / 2) | (uint64_t)(a.d - a.rot);
  auto side = [&](const HeadSide &h) {
    if (!h.heads) return;
    all |= (uint64_t)h.x_ts | (uint64_t)h.x_hs | (uint64_t)h.y_ts | (uint64_t)h.y_hs;
    all |= reinterpret_cast<uintptr_t>(h.x) / esz | reinterpret_cast<uintptr_t>(h.y) / esz;
    all |= reinterpret_cast<uintptr_t>(h.w) / (a.w_f32 ? 4 : 2);
    if (bwd) all |= (uint64_t)h.g_ts | (uint64_t)h.g_hs | reinterpret_cast<uintptr_t>(h.g) / esz;
  };
  side(a.q);
  side(a.k);
  if (a.rot) all |= (reinterpret_cast<uintptr_t>(a.cos) | reinterpret_cast<uintptr_t>(a.sin)) / 4;
  int v = 16 / esz;
  while (v > 1 && all % v) v >>= 1;
  return v;
}

}  // namespace

// Workgroups at most: a few for each of the 256 CUs, each walking over several items so that the weight
// is loaded once for them. 8192 tokens of 32 + 8 heads of 128, whole calls in a row: forward 38.3 us
// with 1024, 35.6 with 1536, 40.6 with 2048 (float32: 62.2, 61.3, 62.6); backward (110 registers, four waves a
// SIMD: 1024 run at once) 62.4 us with 1024, 66.8 with 2048 (float32: 98.1, 105). Two heads at a time a thread
// were slower (registers).
constexpr int kMostFwd = 1536, kMostBwd = 1024;
int head_norm_max_blocks() { return kMostBwd; }   // parts of dw

// Enough workgroups for every item, split between q and k by their heads.
static int head_norm_blocks(int64_t items, int per_block, int64_t most) {
  const int64_t b = (items + per_block - 1) / per_block;
  return (int)(b < most ? b : most);
}

hipError_t launch_head_norm(HeadArgs a, bool f32, bool inter, bool bwd, float *dwq, float *dwk,
                            hipStream_t st) {
  if (a.d < 2 || a.d > 512 || a.rot < 0 || a.rot > a.d || (a.rot & 1) || (a.d & 1)) return hipErrorInvalidValue;
  const int64_t heads = (int64_t)a.q.heads + a.k.heads;
  if (a.m * heads >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  const int vec = chunk_of(a, f32, bwd);
  const int units = a.rot / 2 / vec + ((a.d - a.rot) / vec + 1) / 2;
  int lanes = 1;
  while (lanes < units && lanes < 64) lanes <<= 1;
  a.lanes = lanes;
  const int per_block = kThreads / lanes, most = bwd ? kMostBwd : kMostFwd;
  const int64_t most_q = heads ? (most * (int64_t)a.q.heads + heads - 1) / heads : 0;
  a.blocks_q = a.q.heads ? head_norm_blocks(a.m * a.q.heads, per_block, most_q < most - 1 ? most_q : most - 1) : 0;
  const int blocks_k = a.k.heads ? head_norm_blocks(a.m * a.k.heads, per_block, most - a.blocks_q) : 0;
  const int blocks = a.blocks_q + blocks_k;
  hipError_t e = hipSuccess;
  if (blocks > 0) {
    // a lane holds one unit, or up to four where a head has more than 64 (chunks of one or two)
    if (f32)
      e = vec == 4   ? launch_vec<float, 4, 1>(a, inter, bwd, blocks, st)
          : vec == 2 ? launch_vec<float, 2, 4>(a, inter, bwd, blocks, st)
                     : launch_vec<float, 1, 4>(a, inter, bwd, blocks, st);
    else
      e = vec == 8   ? launch_vec<uint16_t, 8, 1>(a, inter, bwd, blocks, st)
          : vec == 4 ? launch_vec<uint16_t, 4, 1>(a, inter, bwd, blocks, st)
          : vec == 2 ? launch_vec<uint16_t, 2, 4>(a, inter, bwd, blocks, st)
                     : launch_vec<uint16_t, 1, 4>(a, inter, bwd, blocks, st);
    if (e != hipSuccess) return e;
  }
  if (bwd) {
    head_norm_dw_kernel<<<dim3((unsigned)((a.d + kFinCols - 1) / kFinCols), 2), dim3(kFinCols * kFinRows), 0, st>>>(
        a.part, a.d, a.blocks_q, blocks_k, dwq, dwk);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace nf4q
