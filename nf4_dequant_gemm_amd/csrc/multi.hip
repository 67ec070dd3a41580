// Thin products of the layer with an adapter of its own for every row (gfx950, bf16 MFMA): the rows'
// order, T = X A_a^T and U = dY B_a, dA_a = s_a U^T X and dB_a = s_a dY^T T over the rows of adapter
// a, and the transposes they and dX take. The low-rank term of Y and dX is part of the fused kernels
// (multi.h).
//
// Rows are not moved: a table holds them in the order of their adapters and the kernels gather
// through it, so that every 16- or 64-row block has one adapter, whose factor is read once for the
// block. Sums over rows are split into float32 parts that are added in a fixed order.
#include "launch.h"
#include "multi.h"

namespace nf4q {
namespace {

// ------------------------------------------------------------------------------------ row order
// One workgroup: a stable counting sort of the rows by adapter. Wave w counts its run of rows in LDS,
// the counts are scanned over adapters and waves, and each wave then places its rows in order,
// ranking the lanes of equal adapter by a ballot. A wave's ids are loaded eight 64-row pieces at a time.
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64, kPlanAhead = 8;

// Padding of ranks: dst [rows][rp] = src [rows][r] and zeros.
struct PadArgs {
  const uint16_t *src;
  uint16_t *dst;
  int64_t rows;
  int r, rp;
};
__device__ __forceinline__ void pad_rows(const PadArgs &p, int64_t i0, int64_t step) {
  for (int64_t i = i0; i < p.rows * p.rp; i += step) {
    const int64_t row = i / p.rp;
    const int j = (int)(i - row * p.rp);
    p.dst[i] = j < p.r ? p.src[row * p.r + j] : (uint16_t)0;
  }
}

// Workgroups past the first pad the ranks of a factor meanwhile (pad.rows 0: there is none to pad).
__global__ __launch_bounds__(kPlanThreads) void multi_plan_kernel(const int32_t *__restrict__ ids, int64_t M,
                                                                  int L, MultiPlan pl, PadArgs pad) {
  extern __shared__ int32_t cnt[];   // [kPlanWaves][L + 1]
  __shared__ int32_t scan[kMultiTables][kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x > 0) {
    pad_rows(pad, (int64_t)(blockIdx.x - 1) * kPlanThreads + tid, (int64_t)(gridDim.x - 1) * kPlanThreads);
    return;
  }
  const int G = L + 1;
  for (int i = tid; i < kPlanWaves * G; i += kPlanThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t per = ((M + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64;
  const int64_t lo = wave * per, hi = lo + per < M ? lo + per : M;
  volatile int32_t *mine = cnt + wave * G;   // written by one lane, read by the others of its wave
  // groups of the lane's rows i0 + lane, + 64, ... (-1: past the run)
  auto load = [&](int64_t i0, int (&g)[kPlanAhead]) {
    int a[kPlanAhead];
#pragma unroll
    for (int q = 0; q < kPlanAhead; ++q) {
      const int64_t i = i0 + 64 * q + lane;
      a[q] = i < hi ? ids[i] : -1;
    }
#pragma unroll
    for (int q = 0; q < kPlanAhead; ++q) g[q] = i0 + 64 * q + lane >= hi ? -1 : a[q] >= 0 && a[q] < L ? a[q] : L;
  };
  for (int64_t i0 = lo; i0 < hi; i0 += 64 * kPlanAhead) {
    int g[kPlanAhead];
    load(i0, g);
#pragma unroll
    for (int q = 0; q < kPlanAhead; ++q) {   // one addition for each distinct adapter of a piece
      uint64_t left = __ballot(g[q] >= 0);
      while (left) {
        const int a = __builtin_amdgcn_readlane(g[q], __builtin_ctzll(left));
        const uint64_t same = __ballot(g[q] == a);
        if (lane == 0) mine[a] = mine[a] + __popcll(same);
        left &= ~same;
      }
    }
  }
  __syncthreads();
  // adapter g = thread g: its rows and blocks; inclusive scans over the adapters
  int32_t n = 0;
  if (tid < L)
    for (int w = 0; w < kPlanWaves; ++w) n += cnt[w * G + tid];
  int32_t own[kMultiTables], v[kMultiTables];
#pragma unroll
  for (int q = 0; q < kMultiTables; ++q) {
    own[q] = (n + pl.rows[q] - 1) / pl.rows[q];
    scan[q][tid] = own[q];
  }
  __syncthreads();
  for (int o = 1; o < L; o <<= 1) {
#pragma unroll
    for (int q = 0; q < kMultiTables; ++q) v[q] = tid >= o ? scan[q][tid - o] : 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMultiTables; ++q) scan[q][tid] += v[q];
    __syncthreads();
  }
  if (tid < L) {
#pragma unroll
    for (int q = 0; q < kMultiTables; ++q) pl.table[q][tid] = scan[q][tid] - own[q];
    int32_t at = scan[0][tid] - own[0];
    for (int w = 0; w < kPlanWaves; ++w) {
      const int32_t c = cnt[w * G + tid];
      cnt[w * G + tid] = at;
      at += c;
    }
  }
  if (tid == 0) {
    int32_t at = scan[0][L - 1];
    const int32_t none = (int32_t)M - at;
#pragma unroll
    for (int q = 0; q < kMultiTables; ++q) {
      pl.table[q][L] = scan[q][L - 1];
      pl.table[q][L + 1] = scan[q][L - 1] + (none + pl.rows[q] - 1) / pl.rows[q];
    }
    for (int w = 0; w < kPlanWaves; ++w) {
      const int32_t c = cnt[w * G + L];
      cnt[w * G + L] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t i0 = lo; i0 < hi; i0 += 64 * kPlanAhead) {
    int g[kPlanAhead];
    load(i0, g);
#pragma unroll
    for (int q = 0; q < kPlanAhead; ++q) {
      uint64_t left = __ballot(g[q] >= 0);
      while (left) {
        const int a = __builtin_amdgcn_readlane(g[q], __builtin_ctzll(left));
        const uint64_t same = __ballot(g[q] == a);
        const int32_t at = mine[a];   // a wave's LDS accesses are in order
        if (g[q] == a) {
          const int32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
          pl.perm[at + rank] = (int32_t)(i0 + 64 * q + lane);
          if (rank == 0) mine[a] = at + __popcll(same);
        }
        left &= ~same;
      }
    }
  }
}

// The group of block b in a first-block table [L + 2]: every thread tests some groups, the match goes
// through LDS. Called by the whole workgroup; b < first[L + 1].
__device__ __forceinline__ int group_of_block(const int32_t *first, int L, int b) {
  __shared__ int s_group;
  for (int t = threadIdx.x; t <= L; t += blockDim.x)
    if (b >= first[t] && b < first[t + 1]) s_group = t;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(s_group);
}

// ------------------------------------------------------------------------------------ row projection
// part[split][i][j] = sum over the split's l of in[i][l] * p_a[j][l] for the rows i of adapter a and j < r;
// zero for rows without an adapter and for the padding, j < rp. p_a = p + a * pstride, rows of leading
// dimension ldp.

// Blocks of at most 16 rows: latency sets the time, so each wave issues all the loads of a pass
// straight into operand registers. Wave w takes 32-column slices 4 u + w of the workgroup's split
// of the reduction; the four waves' sums are added in wave order in LDS. L % 8 == 0.
template <int TN>
__global__ __launch_bounds__(256) void multi_rows16_kernel(const uint16_t *__restrict__ in, int64_t ldin,
                                                           const uint16_t *__restrict__ p, int64_t pstride,
                                                           int64_t ldp, int64_t M, int64_t Lr, int r, int rp,
                                                           int L, int64_t lsplit, float *__restrict__ part,
                                                           MultiPlan pl) {
  __shared__ f32x4 red[4][TN][64];
  const int b = blockIdx.x;
  if (b >= pl.table[kPlan16][L + 1]) return;
  const int a = group_of_block(pl.table[kPlan16], L, b);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int split = blockIdx.y, nl = lane & 15, kg = lane >> 4;
  const int32_t row0 = pl.table[kPlanRow][a] + (b - pl.table[kPlan16][a]) * 16, rowe = pl.table[kPlanRow][a + 1];
  const bool have = row0 + nl < rowe && a < L;
  const uint16_t *x = in + (have ? (int64_t)pl.perm[row0 + nl] * ldin : 0);
  const uint16_t *pa = p + (a < L ? a : 0) * pstride;
  const int64_t lb = split * lsplit, le = lb + lsplit < Lr ? lb + lsplit : Lr;
  f32x4 acc[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (a < L) {
#pragma unroll 1
    for (int64_t k0 = lb + 32 * wave; k0 < le; k0 += 256) {
      const u32x4 zero = {0u, 0u, 0u, 0u};
      u32x4 xv[2], pv[2][TN];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = k0 + 128 * h + 8 * kg;
        xv[h] = have && c < le ? *reinterpret_cast<const u32x4 *>(x + c) : zero;
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const int j = 16 * t + nl;
          pv[h][t] = j < r && c < le ? *reinterpret_cast<const u32x4 *>(pa + j * ldp + c) : zero;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < TN; ++t)
          acc[t] = mfma16x16x32(__builtin_bit_cast(bf16x8, xv[h]), __builtin_bit_cast(bf16x8, pv[h][t]), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TN; ++t) red[wave][t][lane] = acc[t];
  __syncthreads();
  // D[row][j]: lane l holds column j = l % 16 and rows 4 (l / 16) + v; wave w finishes tiles w, w + 4
  for (int t = wave; t < TN; t += 4) {
    f32x4 s = red[0][t][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) s += red[w][t][lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int32_t row = row0 + 4 * kg + v;
      const int j = 16 * t + nl;
      if (row < rowe && j < rp) part[((int64_t)split * M + pl.perm[row]) * rp + j] = s[v];
    }
  }
}

// Blocks of at most 64 rows (one 16-row tile a wave): in- and p-tiles of 64 columns loaded two steps
// ahead in whole 128-byte rows and staged in LDS, chunk c of row i at slot c ^ ((i >> 1) & 7).
__device__ __forceinline__ int swzm(int row, int c) { return row * 8 + (c ^ ((row >> 1) & 7)); }

template <int TN>
__global__ __launch_bounds__(256) void multi_rows64_kernel(const uint16_t *__restrict__ in, int64_t ldin,
                                                           const uint16_t *__restrict__ p, int64_t pstride,
                                                           int64_t ldp, int64_t M, int64_t Lr, int r, int rp,
                                                           int L, int64_t lsplit, float *__restrict__ part,
                                                           MultiPlan pl) {
  constexpr int PCH = TN * 16 * 8;                 // p-tile chunks per step
  constexpr int PPT = (PCH + 255) / 256;           // p-tile chunks per thread
  __shared__ uint4 sI[2][64 * 8];
  __shared__ uint4 sP[2][PCH];
  const int b = blockIdx.x;
  if (b >= pl.table[kPlan64][L + 1]) return;
  const int a = group_of_block(pl.table[kPlan64], L, b);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int split = blockIdx.y;
  const int32_t row0 = pl.table[kPlanRow][a] + (b - pl.table[kPlan64][a]) * 64, rowe = pl.table[kPlanRow][a + 1];
  const uint16_t *pa = p + (a < L ? a : 0) * pstride;
  const int64_t lb = split * lsplit, le = lb + lsplit < Lr ? lb + lsplit : Lr;
  // this thread's rows of the in-tile (tid / 8 and 32 more), and chunk tid % 8 of each
  const uint16_t *x[2];
  bool have[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t row = row0 + (tid >> 3) + 32 * i;
    have[i] = row < rowe && a < L;
    x[i] = in + (have[i] ? (int64_t)pl.perm[row] * ldin : 0) + (tid & 7) * 8;
  }
  f32x4 acc[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Stage {
    uint4 x[2];
    uint4 q[PPT];
  };
  auto load = [&](int64_t l0, Stage &st) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      st.x[i] = have[i] && l0 + (tid & 7) * 8 < le ? *reinterpret_cast<const uint4 *>(x[i] + l0) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      const int qd = tid + 256 * i;
      const int j = qd >> 3;
      const int64_t l = l0 + (qd & 7) * 8;
      st.q[i] = (qd < PCH && j < r && l < le) ? *reinterpret_cast<const uint4 *>(pa + (int64_t)j * ldp + l)
                                              : make_uint4(0, 0, 0, 0);
    }
  };
  auto store = [&](const Stage &st, int buf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) sI[buf][swzm((tid >> 3) + 32 * i, tid & 7)] = st.x[i];
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      const int qd = tid + 256 * i;
      if (qd < PCH) sP[buf][swzm(qd >> 3, qd & 7)] = st.q[i];
    }
  };
  auto mma = [&](int buf) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int c = kk * 4 + (lane >> 4);
      const bf16x8 xa = __builtin_bit_cast(bf16x8, sI[buf][swzm(wave * 16 + (lane & 15), c)]);
#pragma unroll
      for (int t = 0; t < TN; ++t)
        acc[t] = mfma16x16x32(xa, __builtin_bit_cast(bf16x8, sP[buf][swzm(t * 16 + (lane & 15), c)]), acc[t]);
    }
  };
  Stage s0, s1;
  const int64_t nst = a < L ? (le - lb + 63) / 64 : 0;
  if (nst > 0) load(lb, s0);
  if (nst > 1) load(lb + 64, s1);
  if (nst > 0) store(s0, 0);
  __syncthreads();
  // step i: MFMAs on buffer i & 1; loads of step i + 2; stores of step i + 1 into the other buffer
#pragma unroll 1
  for (int64_t i = 0; i < nst; i += 2) {
    if (i + 2 < nst) load(lb + (i + 2) * 64, s0);
    mma(0);
    if (i + 1 < nst) store(s1, 1);
    __syncthreads();
    if (i + 1 >= nst) break;
    if (i + 3 < nst) load(lb + (i + 3) * 64, s1);
    mma(1);
    if (i + 2 < nst) store(s0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int32_t row = row0 + wave * 16 + 4 * (lane >> 4) + v;
    if (row >= rowe) continue;
    const int64_t i = pl.perm[row];
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const int j = t * 16 + (lane & 15);
      if (j < rp) part[((int64_t)split * M + i) * rp + j] = acc[t][v];
    }
  }
}

// The same product for a batch of at most kMultiSmallM rows without the table of the rows' order
// (multi_rows_of): one workgroup for each 16 rows of an adapter, 32 ranks and slice of the reduction, so
// that a decode step's few adapters are read by many CUs; partial sums [M][r][splits].
__global__ __launch_bounds__(512) void multi_rows_part_kernel(const uint16_t *__restrict__ in, int64_t ldin,
                                                              const uint16_t *__restrict__ p, int64_t pstride,
                                                              int64_t ldp, const int32_t *__restrict__ ids, int M,
                                                              int64_t Lr, int r, int L, float *__restrict__ part) {
  __shared__ __align__(16) uint8_t lds[kMultiSmallT<8, 2>];
  const int splits = gridDim.z, s = blockIdx.z;
  const int64_t per = ((Lr + splits - 1) / splits + 31) / 32 * 32, lb = s * per, le = lb + per < Lr ? lb + per : Lr;
  multi_rows_of<8, 2, 4>(in, ldin, p, pstride, ldp, ids, M, lb, le, r, r, L, blockIdx.x, blockIdx.y * 32, lds,
                         [&](int row, int j, float v) { part[((int64_t)row * r + j) * splits + s] = v; });
}

// bf16(sum over the splits of part [splits][M][rp]), in split order, to out [M][r] and, where the ranks are
// padded, to outp [M][rp].
__global__ void multi_rows_sum_kernel(const float *__restrict__ part, int64_t M, int r, int rp, int splits,
                                      uint16_t *__restrict__ out, uint16_t *__restrict__ outp) {
  const int64_t n = M * rp;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    float a = 0.f;
    int s = 0;
    for (; s + 8 <= splits; s += 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = part[(int64_t)(s + j) * n + i];
#pragma unroll
      for (int j = 0; j < 8; ++j) a += v[j];
    }
    for (; s < splits; ++s) a += part[(int64_t)s * n + i];
    const uint16_t y = (uint16_t)(pack_bf16x2(a, 0.f) & 0xFFFFu);
    if (outp) outp[i] = y;
    if (out) {
      const int64_t row = i / rp;
      const int j = (int)(i - row * rp);
      if (j < r) out[row * r + j] = y;
    }
  }
}

// ------------------------------------------------------------------------------------ sums over rows
// A block of rows (block blockIdx.y of the plan's table `which`, at most kSumRows rows, all of one adapter
// a): the sum over them of P[i][j] * Q[i][c] (dA: P = U, Q = X; dB: P = T, Q = dY), as out holds it
// ([r][C], transposed [C][r]). An adapter of one block writes s[a] times it to out; otherwise it goes to
// part[block] and multi_sum_final_kernel adds the adapter's blocks in order. Blocks of equal size, not a
// split count for every adapter, because one adapter may hold most of the rows.
// Workgroup: 128 columns x all r ranks, in stages of 64 rows loaded two stages ahead, staged row-major
// in LDS (rows padded by 32 bytes) and read with the transposing LDS load, which gives a lane 4
// consecutive rows of one column: the MFMA operand with the rows as its reduction index.
constexpr int kSumRows = 1024;
constexpr int kRB = 64, kCB = 128, kQRow = kCB + 16;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;

__device__ __forceinline__ s16x4 lds_tr(const uint16_t *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}

template <int TJ>
__global__ __launch_bounds__(256) void multi_sum_kernel(const uint16_t *__restrict__ P,
                                                        int64_t ldp, const uint16_t *__restrict__ Q, int64_t ldq,
                                                        int64_t C, int r, int L, int which,
                                                        float *__restrict__ part, const float *__restrict__ s,
                                                        bool transposed, uint16_t *__restrict__ out, MultiPlan pl) {
  constexpr int PROW = TJ * 16 + 16;
  __shared__ uint16_t sQ[2][kRB * kQRow];
  __shared__ uint16_t sP[2][kRB * PROW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * kCB;
  __shared__ int32_t srow[kSumRows];
  const int32_t *first = pl.table[which];
  if ((int)blockIdx.y >= first[L]) return;   // the grid is an upper bound; rows without an adapter add to no sum
  const int a = group_of_block(first, L - 1, blockIdx.y);
  const int nb = first[a + 1] - first[a], size = pl.rows[which];
  const int32_t lo = pl.table[kPlanRow][a] + ((int)blockIdx.y - first[a]) * size;
  const int32_t hi = pl.table[kPlanRow][a + 1];
  const int32_t me = lo + size < hi ? size : hi - lo;   // rows of this block
  for (int i = tid; i < me; i += 256) srow[i] = pl.perm[lo + i];
  __syncthreads();
  f32x4 acc[TJ][2];
#pragma unroll
  for (int t = 0; t < TJ; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Stage {
    uint4 q[4];
    uint4 p[(TJ + 1) / 2];
  };
  auto load = [&](int32_t ms, Stage &st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = tid + 256 * i;
      const int32_t m = ms + (q >> 4);
      const int64_t c = c0 + (q & 15) * 8;
      st.q[i] = (m < me && c < C) ? *reinterpret_cast<const uint4 *>(Q + (int64_t)srow[m] * ldq + c)
                                  : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < (TJ + 1) / 2; ++i) {
      const int q = tid + 256 * i, row = q / (2 * TJ), j = q % (2 * TJ) * 8;
      const int32_t m = ms + row;
      st.p[i] = (row < kRB && m < me && j < r) ? *reinterpret_cast<const uint4 *>(P + (int64_t)srow[m] * ldp + j)
                                               : make_uint4(0, 0, 0, 0);
    }
  };
  auto store = [&](const Stage &st, int buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = tid + 256 * i;
      *reinterpret_cast<uint4 *>(&sQ[buf][(q >> 4) * kQRow + (q & 15) * 8]) = st.q[i];
    }
#pragma unroll
    for (int i = 0; i < (TJ + 1) / 2; ++i) {
      const int q = tid + 256 * i, row = q / (2 * TJ);
      if (row < kRB) *reinterpret_cast<uint4 *>(&sP[buf][row * PROW + q % (2 * TJ) * 8]) = st.p[i];
    }
  };
  const int g16 = lane >> 4, l16 = lane & 15;
  auto frag = [&](const uint16_t *S, int stride, int col0, int ks) {
    const int m0 = ks * 32 + g16 * 8 + (l16 >> 2), col = col0 + 4 * (l16 & 3);
    const s16x4 x = lds_tr(S + m0 * stride + col), y = lds_tr(S + (m0 + 4) * stride + col);
    const s16x8 v = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    return __builtin_bit_cast(bf16x8, v);
  };
  auto mma = [&](int buf) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      bf16x8 q[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) q[u] = frag(sQ[buf], kQRow, wave * 32 + u * 16, ks);
#pragma unroll
      for (int t = 0; t < TJ; ++t) {
        const bf16x8 p = frag(sP[buf], PROW, t * 16, ks);
#pragma unroll
        for (int u = 0; u < 2; ++u) acc[t][u] = mfma16x16x32(p, q[u], acc[t][u]);
      }
    }
  };
  const int nst = (me + kRB - 1) / kRB;
  Stage s0, s1;
  if (nst > 0) load(0, s0);
  if (nst > 1) load(kRB, s1);
  if (nst > 0) store(s0, 0);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < nst; i += 2) {
    if (i + 2 < nst) load((i + 2) * kRB, s0);
    mma(0);
    if (i + 1 < nst) store(s1, 1);
    __syncthreads();
    if (i + 1 >= nst) break;
    if (i + 3 < nst) load((i + 3) * kRB, s1);
    mma(1);
    if (i + 2 < nst) store(s0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < TJ; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int j = t * 16 + 4 * g16 + v;
        const int64_t c = c0 + wave * 32 + u * 16 + l16;
        if (j >= r || c >= C) continue;
        const int64_t at = transposed ? c * r + j : j * C + c;   // as in out
        if (nb > 1)
          part[(int64_t)blockIdx.y * r * C + at] = acc[t][u][v];
        else
          out[(int64_t)a * r * C + at] = (uint16_t)(pack_bf16x2(s[a] * acc[t][u][v], 0.f) & 0xFFFFu);
      }
}

// out[a] = bf16(s[a] * (sum over the adapter's blocks of part)) where the adapter (blockIdx.y) has more
// than one block, zeros where it has none; n values an adapter, two a thread (n is even: r C with
// C % 8 == 0).
__global__ void multi_sum_final_kernel(const float *__restrict__ part, int64_t n, const int32_t *__restrict__ first,
                                       const float *__restrict__ s, uint16_t *__restrict__ out) {
  const int a = blockIdx.y, lo = first[a], nb = first[a + 1] - lo;
  if (nb == 1) return;
  const float sa = s[a];
  for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) * 2; i < n; i += (int64_t)gridDim.x * blockDim.x * 2) {
    const float *pa = part + (int64_t)lo * n + i;
    f32x2 x = {0.f, 0.f};
    int q = 0;
    for (; q + 8 <= nb; q += 8) {
      f32x2 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const f32x2 *>(pa + (int64_t)(q + j) * n);
#pragma unroll
      for (int j = 0; j < 8; ++j) x += v[j];
    }
    for (; q < nb; ++q) x += *reinterpret_cast<const f32x2 *>(pa + (int64_t)q * n);
    *reinterpret_cast<uint32_t *>(out + a * n + i) = nb ? pack_bf16x2(sa * x[0], sa * x[1]) : 0u;
  }
}

// ------------------------------------------------------------------------------------ transposes
// dst[b][c][j] = src[b][j][c] for the bf16 matrices [R][C] of the adapters b that have rows (nobody reads
// the others), of both factors in one launch (blockIdx.z), through 64 x 64 LDS tiles; the rows of dst have ldd elements (a multiple of
// 8), zeros from R on. 16-byte loads where C % 8 == 0, 16-byte stores.
struct TransposeArgs {
  const uint16_t *src;
  uint16_t *dst;
  int64_t R, C, ldd;
};
__global__ __launch_bounds__(256) void multi_transpose_kernel(TransposeArgs b, TransposeArgs a, const int32_t *row) {
  __shared__ uint16_t t[64][66];   // [c][r]
  if (row[blockIdx.y] == row[blockIdx.y + 1]) return;
  const TransposeArgs &g = blockIdx.z ? a : b;
  const int64_t R = g.R, C = g.C, ldd = g.ldd;
  const uint16_t *src = g.src;
  uint16_t *dst = g.dst;
  if ((int64_t)blockIdx.x >= (C + 63) / 64 * ((ldd + 63) / 64)) return;
  const int64_t tiles_c = (C + 63) / 64;
  const int64_t c0 = (int64_t)blockIdx.x % tiles_c * 64, r0 = (int64_t)blockIdx.x / tiles_c * 64;
  src += (int64_t)blockIdx.y * R * C;
  dst += (int64_t)blockIdx.y * ldd * C;
  const int tid = threadIdx.x;
  if ((C & 7) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (tid >> 3) + 32 * h, c = (tid & 7) * 8;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (r0 + r < R && c0 + c < C) v = *reinterpret_cast<const u32x4 *>(src + (r0 + r) * C + c0 + c);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[c + e][r] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    const int x = tid & 63;
    for (int r = tid >> 6; r < 64; r += 4)
      t[x][r] = r0 + r < R && c0 + x < C ? src[(r0 + r) * C + c0 + x] : (uint16_t)0;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = (tid >> 3) + 32 * h, r = (tid & 7) * 8;
    if (c0 + c >= C || r0 + r >= ldd) continue;
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[c][r + 2 * e] | ((uint32_t)t[c][r + 2 * e + 1] << 16);
    *reinterpret_cast<u32x4 *>(dst + (c0 + c) * ldd + r0 + r) = v;
  }
}

__global__ void multi_pad_kernel(PadArgs p) {
  pad_rows(p, blockIdx.x * (int64_t)blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x);
}

int64_t blocks_for(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return b < 4096 ? (b > 0 ? b : 1) : 4096;
}

}  // namespace

hipError_t launch_multi_plan(const int32_t *ids, int64_t M, int L, const MultiPlan &pl, const uint16_t *src, int64_t rows,
                             int r, int rp, uint16_t *dst, hipStream_t st) {
  if (L < 1 || L > kMultiMaxAdapters || M < 1 || M >= (int64_t(1) << 30)) return hipErrorInvalidValue;
  const PadArgs pad{src, dst, r == rp ? 0 : rows, r, rp};
  int64_t blocks = (pad.rows * rp + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  blocks = 1 + (blocks < 1024 ? blocks : 1024);
  multi_plan_kernel<<<dim3((unsigned)blocks), dim3(kPlanThreads), sizeof(int32_t) * kPlanWaves * (L + 1), st>>>(ids, M, L, pl, pad);
  return hipGetLastError();
}

// Rows per block of the row projection: 16 up to 1024 rows, where the groups of a serving batch are a
// few rows each, else 64, which reads an adapter's factor a fourth as often.
static int multi_rows_block(int64_t M) { return M <= 1024 ? 16 : 64; }

// Splits of its reduction: about 1024 workgroups, at least 256 elements each.
int multi_rows_splits(int64_t M, int64_t Lr) {
  const int64_t wgs = (M + multi_rows_block(M) - 1) / multi_rows_block(M);
  int64_t s = (1024 + wgs - 1) / wgs;
  const int64_t most = (Lr + 255) / 256;
  s = s < most ? s : most;
  return (int)(s > 1 ? s : 1);
}

hipError_t launch_multi_rows(const uint16_t *in, int64_t ldin, const uint16_t *p, int64_t pstride, int64_t ldp,
                             int64_t M, int64_t Lr, int r, int rp, int L, int splits, float *part,
                             const MultiPlan &pl, hipStream_t st) {
  const int64_t rows = multi_rows_block(M);
  int64_t lsplit = (Lr + splits - 1) / splits;
  lsplit = (lsplit + 63) / 64 * 64;
  int64_t blocks = (M + (rows - 1) * (L + 1)) / rows;   // >= the sum of ceil(rows of a group / rows)
  blocks = blocks < M ? blocks : M;
  const dim3 grid((unsigned)blocks, (unsigned)splits);
  switch ((r + 15) / 16) {
#define MR_CASE(T)                                                                                                 \
  case T:                                                                                                          \
    if (rows == 16)                                                                                                \
      multi_rows16_kernel<T><<<grid, dim3(256), 0, st>>>(in, ldin, p, pstride, ldp, M, Lr, r, rp, L, lsplit, part, pl); \
    else                                                                                                           \
      multi_rows64_kernel<T><<<grid, dim3(256), 0, st>>>(in, ldin, p, pstride, ldp, M, Lr, r, rp, L, lsplit, part, pl); \
    break;
    MR_CASE(1) MR_CASE(2) MR_CASE(3) MR_CASE(4) MR_CASE(5) MR_CASE(6) MR_CASE(7) MR_CASE(8)
#undef MR_CASE
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_multi_rows_sum(const float *part, int64_t M, int r, int rp, int splits, uint16_t *out, uint16_t *outp,
                                 hipStream_t st) {
  multi_rows_sum_kernel<<<dim3((unsigned)blocks_for(M * rp)), dim3(256), 0, st>>>(part, M, r, rp, splits, out, outp);
  return hipGetLastError();
}

hipError_t launch_multi_rows_part(const uint16_t *in, int64_t ldin, const uint16_t *p, int64_t pstride, int64_t ldp,
                                  const int32_t *ids, int64_t M, int64_t Lr, int r, int L, int splits, float *part,
                                  hipStream_t st) {
  if (M < 1 || M > kMultiSmallM || splits < 1 || splits > 65535) return hipErrorInvalidValue;
  multi_rows_part_kernel<<<dim3((unsigned)M, (unsigned)((r + 31) / 32), (unsigned)splits), dim3(512), 0, st>>>(
      in, ldin, p, pstride, ldp, ids, (int)M, Lr, r, L, part);
  return hipGetLastError();
}

// Rows of a block of the sums over rows: about four workgroups for each of the 256 CUs over the column
// tiles, 64 to 1024 rows.
int multi_sum_rows(int64_t M, int64_t C) {
  const int64_t rows = (M * ((C + kCB - 1) / kCB) / 1024 + kRB - 1) / kRB * kRB;
  return (int)(rows < kRB ? kRB : rows < kSumRows ? rows : kSumRows);
}
int64_t multi_sum_blocks(int64_t M, int64_t C, int L) {
  const int64_t rows = multi_sum_rows(M, C), b = (M + (rows - 1) * L) / rows;   // >= the sum of ceil(rows of a / rows)
  return b < M ? b : M;
}

hipError_t launch_multi_sum(const uint16_t *P, int64_t ldp, const uint16_t *Q, int64_t ldq, int64_t M, int64_t C, int r,
                            int L, const float *s, int which, float *part, uint16_t *out, bool transposed,
                            const MultiPlan &pl, hipStream_t st) {
  const int64_t blocks = multi_sum_blocks(M, C, L);
  if ((ldp & 7) != 0 || ldp < r || (C & 7) != 0 || pl.rows[which] != multi_sum_rows(M, C)) return hipErrorInvalidValue;
  const int64_t tiles = (C + kCB - 1) / kCB;
  if (blocks > 65535) return hipErrorInvalidValue;
  const dim3 grid((unsigned)tiles, (unsigned)blocks);
  switch ((r + 15) / 16) {
#define MS_CASE(T)                                                                                                  case T:                                                                                                             multi_sum_kernel<T><<<grid, dim3(256), 0, st>>>(P, ldp, Q, ldq, C, r, L, which, part, s, transposed, out, pl);     break;
    MS_CASE(1) MS_CASE(2) MS_CASE(3) MS_CASE(4) MS_CASE(5) MS_CASE(6) MS_CASE(7) MS_CASE(8)
#undef MS_CASE
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t n = (int64_t)r * C;
  int64_t b = (n / 2 + 255) / 256;
  b = b < 1024 ? b : 1024;
  multi_sum_final_kernel<<<dim3((unsigned)b, (unsigned)L), dim3(256), 0, st>>>(part, n, pl.table[which], s, out);
  return hipGetLastError();
}

hipError_t launch_multi_transposes(const uint16_t *B, int64_t n, const uint16_t *A, int64_t k, int r, int rp, int L,
                                   const MultiPlan &pl, uint16_t *Bt, uint16_t *At, hipStream_t st) {
  if (rp < r || (rp & 7) != 0 || (n & 7) != 0) return hipErrorInvalidValue;
  const TransposeArgs b{B, Bt, n, r, n}, a{A, At, r, k, rp};
  auto tiles = [](const TransposeArgs &g) { return (g.C + 63) / 64 * ((g.ldd + 63) / 64); };
  const int64_t x = At && tiles(a) > tiles(b) ? tiles(a) : tiles(b);
  multi_transpose_kernel<<<dim3((unsigned)x, (unsigned)L, At ? 2 : 1), dim3(256), 0, st>>>(b, a, pl.table[kPlanRow]);
  return hipGetLastError();
}

hipError_t launch_multi_pad(const uint16_t *src, int64_t rows, int r, int rp, uint16_t *dst, hipStream_t st) {
  const PadArgs p{src, dst, rows, r, rp};
  multi_pad_kernel<<<dim3((unsigned)blocks_for(rows * rp)), dim3(256), 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace nf4q
