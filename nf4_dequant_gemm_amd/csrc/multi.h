// Low-rank term of a GEMM tile whose rows belong to different adapters (device code, shared by the
// fused kernels) and the tables of the rows' order (gfx950).
#pragma once

#include "common.h"

namespace nf4q {

// Row i of the output adds s[a] * P[i] . Q_a[c] with a = ids[i] (none when a lies outside [0, L)):
//   forward: P = T = X A_a^T, Q = B [L][N][r];  dX: P = U = dY B_a, Q = A transposed, [L][K][r].
struct MultiArgs {
  const int32_t *ids;    // [M]
  const float *s;        // [L]
  const uint16_t *P;     // [M][r]
  const uint16_t *Q;     // [L][C][r]
  int L, r;
};

// 8 consecutive ranks j0 .. j0 + 7 of a bf16 row of r ranks starting at element `base` of the
// buffer; ranks at or past r and places past the buffer read as zero. 16-byte loads when the rows are
// 16-byte aligned (r % 8 == 0), else one element at a time.
__device__ __forceinline__ bf16x8 rank_frag(const __amdgpu_buffer_rsrc_t &rs, int64_t base, int j0, int r) {
  u32x4 v;
  if ((r & 7) == 0) {
    v = __builtin_amdgcn_raw_buffer_load_b128(rs, j0 < r ? (uint32_t)((base + j0) * 2) : 0x80000000u, 0, 0);
  } else {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      e[i] = __builtin_amdgcn_raw_buffer_load_b16(rs, j0 + i < r ? (uint32_t)((base + j0 + i) * 2) : 0x80000000u, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (e[2 * i] & 0xFFFFu) | (e[2 * i + 1] << 16);
  }
  return __builtin_bit_cast(bf16x8, v);
}

// The low-rank term of one wave's block of kNT 16-column tiles and kMT 16-row tiles, added to its
// float32 sums acc[nt][mt] (MFMA 16x16x32 with the columns as its first operand: lane (g16, l16)
// holds columns 16 nt + 4 g16 + v of row 16 mt + l16). P and Q are read straight into operand
// registers, once for each 32 ranks: P for the block's rows, then, for each adapter that occurs
// among them (in the order of first occurrence: one for a prompt, up to 16 kMT), Q for the block's
// columns, whose products with the row tiles holding that adapter are added for its rows only.
// The product is scaled in float32. m0, c0: first row and column of the block; rows at or past
// mhi and columns at or past C add nothing.
template <int kNT, int kMT>
__device__ __forceinline__ void multi_term(f32x4 (&acc)[kNT][kMT], const MultiArgs &mu, int64_t m0,
                                           int64_t mhi, int64_t c0, int64_t C) {
  const int lane = threadIdx.x & 63, g16 = lane >> 4, l16 = lane & 15;
  const int r = mu.r;
  int id[kMT];
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt) {
    const int64_t m = m0 + mt * 16 + l16;
    int a = m < mhi ? mu.ids[m] : -1;
    id[mt] = a >= 0 && a < mu.L ? a : -1;
  }
  int64_t rows = mhi - m0;
  rows = rows < 0 ? 0 : rows < 16 * kMT ? rows : 16 * kMT;
  const __amdgpu_buffer_rsrc_t rP = make_rsrc(mu.P + m0 * r, rows * r * 2);
  int64_t cols = C - c0;
  cols = cols < 0 ? 0 : cols < 16 * kNT ? cols : 16 * kNT;
#pragma unroll 1
  for (int j0 = 0; j0 < r; j0 += 32) {
    bf16x8 p[kMT];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) p[mt] = rank_frag(rP, (int64_t)(mt * 16 + l16) * r, j0 + 8 * g16, r);
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
      for (int nt = 0; nt < kNT; ++nt) q[nt] = rank_frag(rQ, (int64_t)(nt * 16 + l16) * r, j0 + 8 * g16, r);
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

// The rows in the order of their adapters (rows without one last, as group L), each group's rows in
// their own order, and each group's first row and first 16- and 64-row block. int32 tables of a
// workspace, written by launch_multi_plan.
constexpr int kMultiMaxAdapters = 1024;
struct MultiPlan {
  int32_t *perm;    // [M]
  int32_t *off;     // [L + 2]
  int32_t *blk16;   // [L + 2]
  int32_t *blk64;   // [L + 2]
};
inline size_t multi_plan_bytes(int64_t m, int L) { return 4 * ((size_t)m + 3 * (size_t)(L + 2)); }
inline MultiPlan multi_plan_at(void *ws, int64_t m, int L) {
  int32_t *p = reinterpret_cast<int32_t *>(ws);
  return MultiPlan{p, p + m, p + m + (L + 2), p + m + 2 * (L + 2)};
}

}  // namespace nf4q
