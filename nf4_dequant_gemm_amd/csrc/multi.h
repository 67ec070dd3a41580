// Low-rank term of a GEMM tile whose rows belong to different adapters (device code, shared by the
// fused kernels) and the tables of the rows' order (gfx950).
#pragma once

#include "common.h"

namespace nf4q {

// Row i of the output adds s[a] * P[i] . Q_a[c] with a = ids[i] (none when a lies outside [0, L)):
//   forward: P = T = X A_a^T, Q = B [L][N][r];  dX: P = U = dY B_a, Q = A transposed, [L][K][r].
// Ranks are padded with zeros to r, a multiple of 8, so that 8 of them are one aligned 16-byte load.
struct MultiArgs {
  const int32_t *ids;    // [M]
  const float *s;        // [L]
  const uint16_t *P;     // [M][r]
  const uint16_t *Q;     // [L][C][r]
  int L, r;
  const int32_t *perm = nullptr;   // [M]: the rows in the order of their adapters, where a kernel takes them so
  // dX with its reduction split over `pieces` workgroups: their float32 sums, [pieces][M][K], which
  // launch_multi_final adds (with the low-rank term)
  int pieces = 1;
  float *part = nullptr;
};
// Bytes of X (dY) that the gathering copies reach with 32-bit offsets; past-the-end rows use an offset
// above it.
constexpr int64_t kMultiMaxGather = 0xFFF00000;

// 8 consecutive ranks j .. j + 7 of row `row` of a bf16 [rows][r] buffer, as an MFMA operand; ranks at or
// past r and rows past the buffer read as zero.
__device__ __forceinline__ bf16x8 rank_frag(const __amdgpu_buffer_rsrc_t &rs, int row, int j, int r) {
  return __builtin_bit_cast(
      bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rs, j < r ? (uint32_t)((row * r + j) * 2) : 0x80000000u, 0, 0));
}

// The low-rank term of one wave's block of kNT 16-column tiles and kMT 16-row tiles, added to its
// float32 sums acc[nt][mt] (MFMA 16x16x32 with the columns as its first operand: lane (g16, l16)
// holds columns 16 nt + 4 g16 + v of row 16 mt + l16). P and Q go straight to operand registers, for
// 32 ranks at a time: P for the block's rows, then, for each adapter that occurs among them (in the
// order of first occurrence), Q for the block's columns, whose products with the row tiles that hold
// the adapter are added for its rows only, scaled in float32. Rows come in the order of their adapters
// (perm), so that a block rarely has more than two. Row m of the block's order is row perm[m] of P and
// ids (perm NULL: row m); m0, c0: first row and column of the block; rows at or past mhi and columns
// at or past C add nothing.
template <int kNT, int kMT>
__device__ __forceinline__ void multi_term(f32x4 (&acc)[kNT][kMT], const MultiArgs &mu, const int32_t *perm,
                                           int64_t m0, int64_t mhi, int64_t c0, int64_t C) {
  const int lane = threadIdx.x & 63, g16 = lane >> 4, l16 = lane & 15;
  const int r = mu.r;
  int id[kMT];
  int64_t at[kMT];
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt) {
    const int64_t m = m0 + mt * 16 + l16;
    at[mt] = m < mhi ? (perm ? perm[m] : m) : -1;
    const int a = m < mhi ? mu.ids[at[mt]] : -1;
    id[mt] = a >= 0 && a < mu.L ? a : -1;
  }
  int64_t cols = C - c0;
  cols = cols < 0 ? 0 : cols < 16 * kNT ? cols : 16 * kNT;
#pragma unroll 1
  for (int j0 = 0; j0 < r; j0 += 32) {
    bf16x8 p[kMT];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (id[mt] >= 0 && j0 + 8 * g16 < r) v = *reinterpret_cast<const u32x4 *>(mu.P + at[mt] * r + j0 + 8 * g16);
      p[mt] = __builtin_bit_cast(bf16x8, v);
    }
    uint32_t left = 0;   // row tiles whose row of this lane still waits for its adapter
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) left |= id[mt] >= 0 ? 1u << mt : 0u;
#pragma unroll 1
    while (true) {
      const uint64_t who = __ballot(left != 0);
      if (!who) break;
      int first = 0;
#pragma unroll
      for (int mt = kMT - 1; mt >= 0; --mt) first = (left >> mt) & 1 ? id[mt] : first;
      const int a = __builtin_amdgcn_readlane(first, __builtin_ctzll(who));
      const float sa = mu.s[a];
      const __amdgpu_buffer_rsrc_t rQ = make_rsrc(mu.Q + ((int64_t)a * C + c0) * r, cols * r * 2);
      bf16x8 q[kNT];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) q[nt] = rank_frag(rQ, nt * 16 + l16, j0 + 8 * g16, r);
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const bool mine = id[mt] == a;
        if (__ballot(mine)) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            const f32x4 d = mfma16x16x32(q[nt], p[mt], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[nt][mt][v] += mine ? sa * d[v] : 0.f;
          }
          if (mine) left &= ~(1u << mt);
        }
      }
    }
  }
}

// The same for one row tile of a serving batch, where every row may have an adapter of its own: Q of up
// to kB of them is requested together (one round trip to memory for each would be the whole time of
// the term: 16 adapters took 16 us). load_p(rank) gives a lane its 8 ranks of row l16; id is that row's
// adapter or -1.
template <int kB, int kNT, typename LoadP>
__device__ __forceinline__ void multi_term_rows(f32x4 (&acc)[kNT], const MultiArgs &mu, int id, int64_t c0, int64_t C,
                                                LoadP load_p) {
  const int lane = threadIdx.x & 63, g16 = lane >> 4, l16 = lane & 15;
  const int r = mu.r;
  int64_t cols = C - c0;
  cols = cols < 0 ? 0 : cols < 16 * kNT ? cols : 16 * kNT;
#pragma unroll 1
  for (int j0 = 0; j0 < r; j0 += 32) {
    const bf16x8 p = load_p(j0 + 8 * g16);
    uint64_t left = __ballot(id >= 0);
#pragma unroll 1
    while (left) {
      int a[kB];
      float sa[kB];
      bf16x8 q[kB][kNT];
#pragma unroll
      for (int e = 0; e < kB; ++e) {
        a[e] = left ? __builtin_amdgcn_readlane(id, __builtin_ctzll(left)) : -2;   // -2: no row's
        left &= ~__ballot(id == a[e]);
        const int at = a[e] < 0 ? 0 : a[e];
        sa[e] = mu.s[at];
        const __amdgpu_buffer_rsrc_t rQ =
            make_rsrc(mu.Q + ((int64_t)at * C + c0) * r, a[e] < 0 ? 0 : cols * r * 2);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) q[e][nt] = rank_frag(rQ, nt * 16 + l16, j0 + 8 * g16, r);
      }
#pragma unroll
      for (int e = 0; e < kB; ++e) {
        const bool mine = id == a[e];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const f32x4 d = mfma16x16x32(q[e][nt], p, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[nt][v] += mine ? sa[e] * d[v] : 0.f;
        }
      }
    }
  }
}

// ---- T = X A_a^T of a batch of at most kMultiSmallM rows, without the table of the rows' order, by one
// workgroup of kW waves for its slice of the reduction: `row` is the row it stands for, and it stands
// down unless that is the first, seventeenth, ... row of its adapter; it then takes that row and the
// adapter's next ones, up to 16, and the 16 TN ranks from j0. Each wave's loads for kU slices of 32 go
// straight to operand registers before their MFMAs; the waves' sums are added in wave order in LDS
// and handed to put(row, rank, sum) for ranks below rp, zeros past r (a row without an adapter: all
// zeros). lds: kMultiSmallT bytes.
constexpr int kMultiSmallM = 256;   // rows
template <int kW, int TN>
constexpr int kMultiSmallT = kW * TN * 64 * 16 + (kMultiSmallM / 64) * 8 + 16 * 4;
template <int kW, int TN, int kU, typename Put>
__device__ __forceinline__ void multi_rows_of(const uint16_t *in, int64_t ldin, const uint16_t *p, int64_t pstride,
                                              int64_t ldp, const int32_t *ids, int M, int64_t lb, int64_t le, int r,
                                              int rp, int L, int row, int j0, void *lds, Put put) {
  f32x4 *red = reinterpret_cast<f32x4 *>(lds);                      // [kW][TN][64]
  uint64_t *same = reinterpret_cast<uint64_t *>(red + kW * TN * 64);
  int *rows = reinterpret_cast<int *>(same + kMultiSmallM / 64);
  static_assert(kW >= kMultiSmallM / 64, "a lane for every row");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto clip = [&](int a) { return a >= 0 && a < L ? a : -1; };
  const int a = __builtin_amdgcn_readfirstlane(clip(ids[row]));
  bool match = false;
  if (wave < kMultiSmallM / 64) {
    match = tid < M && clip(ids[tid]) == a;
    const uint64_t b = __ballot(match);
    if (lane == 0) same[wave] = b;
  }
  __syncthreads();
  auto before = [&](int i) {   // rows of this adapter before row i
    int n = 0;
#pragma unroll
    for (int w = 0; w < kMultiSmallM / 64; ++w) {
      const uint64_t m = i >= 64 * (w + 1) ? ~uint64_t(0) : i <= 64 * w ? 0 : (uint64_t(1) << (i - 64 * w)) - 1;
      n += __popcll(same[w] & m);
    }
    return n;
  };
  const int first = before(row);
  if (first % 16) return;
  const int all = before(kMultiSmallM);
  const int n = all - first < 16 ? all - first : 16;
  if (match) {
    const int q = before(tid) - first;
    if (q >= 0 && q < 16) rows[q] = tid;
  }
  __syncthreads();
  const int nl = lane & 15, kg = lane >> 4;
  f32x4 acc[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (a >= 0) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const bool have = nl < n;
    const uint16_t *x = in + (have ? rows[nl] * ldin : 0);
    const uint16_t *pa = p + a * pstride;
#pragma unroll 1
    for (int64_t k0 = lb + 32 * wave + 8 * kg; k0 < le; k0 += kU * 32 * kW) {
      u32x4 xv[kU], pv[kU][TN];
#pragma unroll
      for (int h = 0; h < kU; ++h) {
        const int64_t c = k0 + h * 32 * kW;
        xv[h] = have && c < le ? *reinterpret_cast<const u32x4 *>(x + c) : zero;
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const int j = j0 + 16 * t + nl;
          pv[h][t] = j < r && c < le ? *reinterpret_cast<const u32x4 *>(pa + j * ldp + c) : zero;
        }
      }
#pragma unroll
      for (int h = 0; h < kU; ++h)
#pragma unroll
        for (int t = 0; t < TN; ++t)
          acc[t] = mfma16x16x32(__builtin_bit_cast(bf16x8, xv[h]), __builtin_bit_cast(bf16x8, pv[h][t]), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TN; ++t) red[(wave * TN + t) * 64 + lane] = acc[t];
  __syncthreads();
  if (wave < TN) {
    f32x4 s = red[wave * 64 + lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) s += red[(w * TN + wave) * 64 + lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int q = 4 * kg + v, j = j0 + 16 * wave + nl;
      if (q < n && j < rp) put(rows[q], j, s[v]);
    }
  }
}

// The rows in the order of their adapters (rows without one last, as group L), each group's rows in
// their own order, and each group's first row and first block of 16 rows, of 64 rows, and of the rows
// that the sums over rows take at a time. int32 tables of a workspace, written by launch_multi_plan.
constexpr int kMultiMaxAdapters = 1024;
constexpr int kMultiTables = 4;
struct MultiPlan {
  int32_t *perm;                 // [M]
  int32_t *table[kMultiTables];  // [L + 2] each: first row, then first blocks
  int rows[kMultiTables];        // rows of a block: 1, 16, 64, and the sums'
};
enum { kPlanRow = 0, kPlan16 = 1, kPlan64 = 2, kPlanSum = 3 };
inline size_t multi_plan_bytes(int64_t m, int L) { return 4 * ((size_t)m + kMultiTables * (size_t)(L + 2)); }
inline MultiPlan multi_plan_at(void *ws, int64_t m, int L, int sum_rows) {
  int32_t *p = reinterpret_cast<int32_t *>(ws);
  MultiPlan pl{p, {}, {1, 16, 64, sum_rows}};
  for (int t = 0; t < kMultiTables; ++t) pl.table[t] = p + m + t * (L + 2);
  return pl;
}

}  // namespace nf4q
