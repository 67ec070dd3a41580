// Thin products of the layer with an adapter of its own for every row (gfx950, bf16 MFMA): the rows'
// order, T = X A_a^T and U = dY B_a, dA_a = s_a U^T X and dB_a = s_a dY^T T over the rows of adapter
// a, and the transposes they and dX take. The low-rank term of Y and dX is part of the fused kernels
// (multi.h).
//
// Rows are not moved: a table holds them in the order of their adapters and the kernels gather
// through it, so that every 16- or 64-row block has one adapter, whose factor is read once for the
// block. Sums over rows are split into float32 parts that are added in a fixed order.
#include <algorithm>
#include <cmath>

#include "launch.h"
#include "multi.h"

namespace nf4q {
namespace {

// ------------------------------------------------------------------------------------ row order
// One workgroup: a stable counting sort of the rows by adapter. Wave w counts its run of rows in LDS,
// the counts are scanned over adapters and waves, and each wave then places its rows in order. The
// lanes of a 64-row piece are ranked within their adapter by ballots, one for each adapter in the
// piece, so that LDS is read and written once a piece. A wave's ids are loaded eight pieces at a time.
// Bound by latency (two passes over the ids, a scan, barriers): 500 rows 6.2 us, 4096 rows 8.4, 8192 rows 9.4.
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

// dst[a][c][j] = src[a][j][c] of the bf16 matrices [R][C] of an adapter a that has rows (nobody reads the
// others), through LDS tiles of 4096 elements, four to a workgroup; the rows of dst have ldd elements (a
// multiple of 8), zeros from R on. 16-byte loads where C % 8 == 0, 16-byte stores. A tile is as wide as
// the rank (8, 16, 32 or 64) and takes more of the long side instead: square ones left 60 adapters of rank 8
// x 4096 seven eighths empty and took 18 us; 8 x 8 elements a thread in registers, without LDS, were
// 4 to 26 us slower (scattered 16-byte loads of few workgroups).
struct TransposeArgs {
  const uint16_t *src;
  uint16_t *dst;
  int64_t R, C, ldd;
  int lr, lc;   // log2 of a tile's rows and columns: lr + lc = 12, each at least 3
  __host__ __device__ int64_t tiles_r() const { return (ldd + (1 << lr) - 1) >> lr; }
  __host__ __device__ int64_t tiles_c() const { return (C + (1 << lc) - 1) >> lc; }
  __host__ __device__ int64_t blocks() const { return src ? (tiles_r() * tiles_c() + 3) / 4 : 0; }
};
constexpr int kTileLds = 4096 + 512;   // its columns, each padded by one (an even stride: 16 lanes on a bank)
// log2 of a tile's extent along ranks
int rank_log(int r) { return r <= 8 ? 3 : r <= 16 ? 4 : r <= 32 ? 5 : 6; }
// Rows that are looked through for an adapter's use; one that they do not show in a longer batch is
// transposed unused.
constexpr int64_t kUseRows = 8192;
__device__ __forceinline__ void transpose_tiles(const TransposeArgs &g, const int32_t *ids, int64_t M, int a,
                                                int64_t block, uint16_t (&lds)[4][kTileLds]) {
  bool used = M > kUseRows;
  for (int64_t i0 = threadIdx.x; i0 < M && i0 < kUseRows; i0 += kPlanThreads) used |= ids[i0] == a;
  if (!__syncthreads_or(used)) return;
  const int tid = threadIdx.x & 255, stride = (1 << g.lr) + 1;
  const int64_t tile = block * 4 + (threadIdx.x >> 8), tiles_c = g.tiles_c();
  const int64_t c0 = (tile % tiles_c) << g.lc, r0 = (tile / tiles_c) << g.lr;
  const bool mine = r0 < g.ldd;
  uint16_t *t = lds[threadIdx.x >> 8];   // [c][r]
  const uint16_t *src = g.src + (int64_t)a * g.R * g.C;
  uint16_t *dst = g.dst + (int64_t)a * g.ldd * g.C;
  if (!mine) {
  } else if ((g.C & 7) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int q = tid + 256 * h, r = q >> (g.lc - 3), c = (q & ((1 << (g.lc - 3)) - 1)) * 8;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (r0 + r < g.R && c0 + c < g.C) v = *reinterpret_cast<const u32x4 *>(src + (r0 + r) * g.C + c0 + c);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[(c + e) * stride + r] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  } else {
#pragma unroll
    for (int h = 0; h < 16; ++h) {
      const int q = tid + 256 * h, r = q >> g.lc, c = q & ((1 << g.lc) - 1);
      t[c * stride + r] = r0 + r < g.R && c0 + c < g.C ? src[(r0 + r) * g.C + c0 + c] : (uint16_t)0;
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int q = tid + 256 * h, c = q >> (g.lr - 3), r = (q & ((1 << (g.lr - 3)) - 1)) * 8;
    if (!mine || c0 + c >= g.C || r0 + r >= g.ldd) continue;
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[c * stride + r + 2 * e] | ((uint32_t)t[c * stride + r + 2 * e + 1] << 16);
    *reinterpret_cast<u32x4 *>(dst + (c0 + c) * g.ldd + r0 + r) = v;
  }
}

// The first workgroup orders the rows, which leaves the card idle for 6 to 9 us; the others meanwhile pad the
// ranks of a factor (pad.rows 0: there is none to pad) and transpose the adapters for the backward.
struct PlanWork {
  PadArgs pad;
  int pad_blocks;
  TransposeArgs tr[2];
};
__global__ __launch_bounds__(kPlanThreads) void multi_plan_kernel(const int32_t *__restrict__ ids, int64_t M,
                                                                  int L, MultiPlan pl, PlanWork work) {
  extern __shared__ int32_t cnt[];   // [kPlanWaves][L + 1]
  __shared__ int32_t scan[kMultiTables][kPlanThreads];
  __shared__ __align__(16) uint16_t tile[4][kTileLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x > 0) {
    int64_t b = (int64_t)blockIdx.x - 1;
    if (b < work.pad_blocks) {
      pad_rows(work.pad, b * kPlanThreads + tid, (int64_t)work.pad_blocks * kPlanThreads);
      return;
    }
    b -= work.pad_blocks;
    const bool second = b >= work.tr[0].blocks() * L;
    if (second) b -= work.tr[0].blocks() * L;
    const TransposeArgs g = second ? work.tr[1] : work.tr[0];
    transpose_tiles(g, ids, M, (int)(b / g.blocks()), b % g.blocks(), tile);
    return;
  }
  const int G = L + 1;
  for (int i = tid; i < kPlanWaves * G; i += kPlanThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t per = ((M + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64;
  const int64_t lo = wave * per, hi = lo + per < M ? lo + per : M;
  volatile int32_t *mine = cnt + wave * G;   // a wave's LDS accesses are in order
  // groups of the lane's rows i0 + lane, + 64, ... (-1: past the run)
  int g[kPlanAhead];
  auto load = [&](int64_t i0) {
    int a[kPlanAhead];
#pragma unroll
    for (int q = 0; q < kPlanAhead; ++q) {
      const int64_t i = i0 + 64 * q + lane;
      a[q] = i < hi ? ids[i] : -1;
    }
#pragma unroll
    for (int q = 0; q < kPlanAhead; ++q) g[q] = i0 + 64 * q + lane >= hi ? -1 : a[q] >= 0 && a[q] < L ? a[q] : L;
  };
  // the lane's rank among the piece's rows of its group, and their number
  auto rank_of = [&](int group, int &rank, int &rows) {
    rank = rows = 0;
    for (uint64_t left = __ballot(group >= 0); left;) {
      const int a = __builtin_amdgcn_readlane(group, __builtin_ctzll(left));
      const uint64_t same = __ballot(group == a);
      if (group == a) {
        rank = __popcll(same & ((uint64_t(1) << lane) - 1));
        rows = __popcll(same);
      }
      left &= ~same;
    }
  };
  for (int64_t i0 = lo; i0 < hi; i0 += 64 * kPlanAhead) {
    load(i0);
#pragma unroll
    for (int q = 0; q < kPlanAhead; ++q) {
      int rank, rows;
      rank_of(g[q], rank, rows);
      if (g[q] >= 0 && rank == 0) mine[g[q]] = mine[g[q]] + rows;
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
  // a group's first place in every wave's run, from its first place
  auto place = [&](int group, int32_t at) {
    int32_t c[kPlanWaves];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) c[w] = cnt[w * G + group];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      cnt[w * G + group] = at;
      at += c[w];
    }
  };
  if (tid < L) {
#pragma unroll
    for (int q = 0; q < kMultiTables; ++q) pl.table[q][tid] = scan[q][tid] - own[q];
    place(tid, scan[0][tid] - own[0]);
  }
  if (tid == 0) {
    int32_t at = scan[0][L - 1];
    const int32_t none = (int32_t)M - at;
#pragma unroll
    for (int q = 0; q < kMultiTables; ++q) {
      pl.table[q][L] = scan[q][L - 1];
      pl.table[q][L + 1] = scan[q][L - 1] + (none + pl.rows[q] - 1) / pl.rows[q];
    }
    place(L, at);
  }
  __syncthreads();
  for (int64_t i0 = lo; i0 < hi; i0 += 64 * kPlanAhead) {
    if (per > 64 * kPlanAhead) load(i0);   // else they are still here
#pragma unroll
    for (int q = 0; q < kPlanAhead; ++q) {
      int rank, rows;
      rank_of(g[q], rank, rows);
      if (g[q] < 0) continue;
      const int32_t at = mine[g[q]];
      pl.perm[at + rank] = (int32_t)(i0 + 64 * q + lane);
      if (rank == 0) mine[g[q]] = at + rows;
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
// MultiRows (launch.h): part[split][i][j] = sum over the split's l of in[i][l] * p_a[j][l] for the rows i of
// adapter a and j < r; zero for rows without an adapter and for the padding, j < rp. Up to two products
// in a launch (blockIdx.z).
struct RowsArgs {
  MultiRows g[2];
  int64_t lsplit[2], M;
  int r, rp, L;
};

// Blocks of at most 16 rows: latency sets the time, so each wave issues all the loads of a pass
// straight into operand registers. Wave w takes 32-column slices 4 u + w of the workgroup's split
// of the reduction; the four waves' sums are added in wave order in LDS. L % 8 == 0.
template <int TN>
__global__ __launch_bounds__(256) void multi_rows16_kernel(RowsArgs w, MultiPlan pl) {
  __shared__ f32x4 red[4][TN][64];
  const int b = blockIdx.x, split = blockIdx.y, L = w.L, r = w.r, rp = w.rp;
  const MultiRows g = blockIdx.z ? w.g[1] : w.g[0];
  if (split >= g.splits || b >= pl.table[kPlan16][L + 1]) return;
  const int a = group_of_block(pl.table[kPlan16], L, b);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nl = lane & 15, kg = lane >> 4;
  const int32_t row0 = pl.table[kPlanRow][a] + (b - pl.table[kPlan16][a]) * 16, rowe = pl.table[kPlanRow][a + 1];
  const bool have = row0 + nl < rowe && a < L;
  const uint16_t *x = g.in + (have ? (int64_t)pl.perm[row0 + nl] * g.l : 0);
  const uint16_t *pa = g.p + (int64_t)(a < L ? a : 0) * r * g.l;
  const int64_t lsplit = blockIdx.z ? w.lsplit[1] : w.lsplit[0];
  const int64_t lb = split * lsplit, le = lb + lsplit < g.l ? lb + lsplit : g.l;
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
          pv[h][t] = j < r && c < le ? *reinterpret_cast<const u32x4 *>(pa + j * g.l + c) : zero;
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
    for (int q = 1; q < 4; ++q) s += red[q][t][lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int32_t row = row0 + 4 * kg + v;
      const int j = 16 * t + nl;
      if (row < rowe && j < rp) g.part[((int64_t)split * w.M + pl.perm[row]) * rp + j] = s[v];
    }
  }
}

// Blocks of at most 64 rows (one 16-row tile a wave): in- and p-tiles of 64 columns loaded two steps
// ahead in whole 128-byte rows and staged in LDS, chunk c of row i at slot c ^ ((i >> 1) & 7). Bound by its
// loads: 8192 rows of 4 adapters, r 64, 4096 columns 22 us (3.1 TB/s), 11008 columns 50 us (3.6 TB/s).
__device__ __forceinline__ int swzm(int row, int c) { return row * 8 + (c ^ ((row >> 1) & 7)); }

template <int TN>
__global__ __launch_bounds__(256) void multi_rows64_kernel(RowsArgs w, MultiPlan pl) {
  constexpr int PCH = TN * 16 * 8;                 // p-tile chunks per step
  constexpr int PPT = (PCH + 255) / 256;           // p-tile chunks per thread
  __shared__ uint4 sI[2][64 * 8];
  __shared__ uint4 sP[2][PCH];
  const int b = blockIdx.x, split = blockIdx.y, L = w.L, r = w.r, rp = w.rp;
  const MultiRows g = blockIdx.z ? w.g[1] : w.g[0];
  if (split >= g.splits || b >= pl.table[kPlan64][L + 1]) return;
  const int a = group_of_block(pl.table[kPlan64], L, b);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t row0 = pl.table[kPlanRow][a] + (b - pl.table[kPlan64][a]) * 64, rowe = pl.table[kPlanRow][a + 1];
  const uint16_t *pa = g.p + (int64_t)(a < L ? a : 0) * r * g.l;
  const int64_t lsplit = blockIdx.z ? w.lsplit[1] : w.lsplit[0];
  const int64_t lb = split * lsplit, le = lb + lsplit < g.l ? lb + lsplit : g.l;
  // this thread's rows of the in-tile (tid / 8 and 32 more), and chunk tid % 8 of each
  const uint16_t *x[2];
  bool have[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t row = row0 + (tid >> 3) + 32 * i;
    have[i] = row < rowe && a < L;
    x[i] = g.in + (have[i] ? (int64_t)pl.perm[row] * g.l : 0) + (tid & 7) * 8;
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
      st.q[i] = (qd < PCH && j < r && l < le) ? *reinterpret_cast<const uint4 *>(pa + (int64_t)j * g.l + l)
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
      if (j < rp) g.part[((int64_t)split * w.M + i) * rp + j] = acc[t][v];
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

// The sum over the splits of part [splits][M][rp], in split order, in bf16 to out [M][r] and padded [M][rp] and
// in float32 to wide [M][rp], each where it is given.
__global__ void multi_rows_sum_kernel(RowsArgs w) {
  const MultiRows g = blockIdx.y ? w.g[1] : w.g[0];
  const int64_t n = w.M * w.rp;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    float a = 0.f;
    int s = 0;
    for (; s + 8 <= g.splits; s += 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = g.part[(int64_t)(s + j) * n + i];
#pragma unroll
      for (int j = 0; j < 8; ++j) a += v[j];
    }
    for (; s < g.splits; ++s) a += g.part[(int64_t)s * n + i];
    const uint16_t y = (uint16_t)(pack_bf16x2(a, 0.f) & 0xFFFFu);
    if (g.padded) g.padded[i] = y;
    if (g.wide) g.wide[i] = a;
    if (g.out) {
      const int64_t row = i / w.rp;
      const int j = (int)(i - row * w.rp);
      if (j < w.r) g.out[row * w.r + j] = y;
    }
  }
}

// ------------------------------------------------------------------------------------ sums over rows
// dA and dB in one launch (blockIdx.z). A block of rows (block blockIdx.y of the plan's table kPlanSum, at
// most kSumRows rows, all of one adapter a): the sum over them of P[i][j] * Q[i][c] (dA: P = U, Q = X; dB:
// P = T, Q = dY), as out holds it ([r][C], transposed [C][r]). An adapter of one block writes s[a] times
// it to out; otherwise it goes to part[block] and multi_sum_final_kernel adds the adapter's blocks in
// order. Blocks of equal size, not a split count for every adapter, because one adapter may hold most of
// the rows. At most kMultiSmallM rows (kSmall): a block is an adapter, which writes its zeros too, and P
// is float32, taken as the sum of two bf16 numbers (16 bits of mantissa): the products are few, and with
// one row to an adapter P's rounding to bf16 would be half the error of dA and dB.
// Workgroup: 128 columns x all r ranks, in stages of kR = 64 rows loaded two stages ahead, staged row-major
// in LDS (rows padded by 32 bytes) and read with the transposing LDS load, which gives a lane 4
// consecutive rows of one column: the MFMA operand with the rows as its reduction index. dA and dB of 8192
// rows of 4 adapters, r 64, 4096 and 11008 columns: 62 us (4 TB/s of X and dY) and 14 us to add the blocks.
constexpr int kSumRows = 1024;
constexpr int kRB = 64, kCB = 128, kQRow = kCB + 16;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;

__device__ __forceinline__ s16x4 lds_tr(const uint16_t *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}

struct SumArgs {
  MultiSum g[2];
  const float *s;
  int r, rp, L;
};

template <int TJ, bool kSmall, int kR>
__global__ __launch_bounds__(256) void multi_sum_kernel(SumArgs w, MultiPlan pl) {
  constexpr int PROW = TJ * 16 + 16, kParts = kSmall ? 2 : 1;
  constexpr int kPI = (kR * 2 * TJ + 255) / 256;   // 8-rank pieces of a thread
  __shared__ __align__(16) uint16_t sQ[2][kR * kQRow];
  __shared__ __align__(16) uint16_t sP[2][kParts][kR * PROW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = w.r;
  const MultiSum g = blockIdx.z ? w.g[1] : w.g[0];
  const int64_t c0 = (int64_t)blockIdx.x * kCB, C = g.c;
  if (c0 >= C) return;
  __shared__ int32_t srow[kSmall ? kMultiSmallM : kSumRows];
  int a = blockIdx.y, nb = 1;
  int32_t lo, me;   // first row of this block, and its rows
  if constexpr (kSmall) {
    lo = pl.table[kPlanRow][a];
    me = pl.table[kPlanRow][a + 1] - lo;
  } else {
    const int32_t *first = pl.table[kPlanSum];
    if ((int)blockIdx.y >= first[w.L]) return;   // the grid is an upper bound; rows without an adapter add to no sum
    a = group_of_block(first, w.L - 1, blockIdx.y);
    nb = first[a + 1] - first[a];
    const int size = pl.rows[kPlanSum];
    lo = pl.table[kPlanRow][a] + ((int)blockIdx.y - first[a]) * size;
    const int32_t hi = pl.table[kPlanRow][a + 1];
    me = lo + size < hi ? size : hi - lo;
  }
  for (int i = tid; i < me; i += 256) srow[i] = pl.perm[lo + i];
  __syncthreads();
  f32x4 acc[TJ][2];
#pragma unroll
  for (int t = 0; t < TJ; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Stage {
    uint4 q[kR / 16];
    uint4 p[kPI][kParts];   // 8 ranks, in bf16 or float32
  };
  auto load = [&](int32_t ms, Stage &st) {
#pragma unroll
    for (int i = 0; i < kR / 16; ++i) {
      const int q = tid + 256 * i;
      const int32_t m = ms + (q >> 4);
      const int64_t c = c0 + (q & 15) * 8;
      st.q[i] = (m < me && c < C) ? *reinterpret_cast<const uint4 *>(g.q + (int64_t)srow[m] * C + c)
                                  : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kPI; ++i) {
      const int q = tid + 256 * i, row = q / (2 * TJ), j = q % (2 * TJ) * 8;
      const int32_t m = ms + row;
      const bool have = row < kR && m < me && j < r;
#pragma unroll
      for (int e = 0; e < kParts; ++e)
        st.p[i][e] = have ? reinterpret_cast<const uint4 *>((const uint16_t *)g.p +
                                                            ((int64_t)srow[m] * w.rp + j) * kParts)[e]
                          : make_uint4(0, 0, 0, 0);
    }
  };
  auto store = [&](const Stage &st, int buf) {
#pragma unroll
    for (int i = 0; i < kR / 16; ++i) {
      const int q = tid + 256 * i;
      *reinterpret_cast<uint4 *>(&sQ[buf][(q >> 4) * kQRow + (q & 15) * 8]) = st.q[i];
    }
#pragma unroll
    for (int i = 0; i < kPI; ++i) {
      const int q = tid + 256 * i, row = q / (2 * TJ);
      if (row >= kR) continue;
      uint16_t *at = &sP[buf][0][row * PROW + q % (2 * TJ) * 8];
      if constexpr (kSmall) {
        const float *v = reinterpret_cast<const float *>(&st.p[i][0]);
        uint32_t hi[4], rest[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hi[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
          const float x = __builtin_bit_cast(float, hi[e] << 16), y = __builtin_bit_cast(float, hi[e] & 0xFFFF0000u);
          // nothing is left of an infinity
          rest[e] = pack_bf16x2(fabsf(x) < INFINITY ? v[2 * e] - x : 0.f, fabsf(y) < INFINITY ? v[2 * e + 1] - y : 0.f);
        }
        *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(at + kR * PROW) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
      } else {
        *reinterpret_cast<uint4 *>(at) = st.p[i][0];
      }
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
    for (int ks = 0; ks < kR / 32; ++ks) {
      bf16x8 q[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) q[u] = frag(sQ[buf], kQRow, wave * 32 + u * 16, ks);
#pragma unroll
      for (int t = 0; t < TJ; ++t) {
#pragma unroll
        for (int e = 0; e < kParts; ++e) {
          const bf16x8 p = frag(sP[buf][e], PROW, t * 16, ks);
          // the operand whose index runs along out's rows comes first: a lane then holds 4 of them
          if (g.transposed) {
#pragma unroll
            for (int u = 0; u < 2; ++u) acc[t][u] = mfma16x16x32(p, q[u], acc[t][u]);
          } else {
#pragma unroll
            for (int u = 0; u < 2; ++u) acc[t][u] = mfma16x16x32(q[u], p, acc[t][u]);
          }
        }
      }
    }
  };
  const int nst = (me + kR - 1) / kR;
  Stage s0, s1;
  if (nst > 0) load(0, s0);
  if (nst > 1) load(kR, s1);
  if (nst > 0) store(s0, 0);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < nst; i += 2) {
    if (i + 2 < nst) load((i + 2) * kR, s0);
    mma(0);
    if (i + 1 < nst) store(s1, 1);
    __syncthreads();
    if (i + 1 >= nst) break;
    if (i + 3 < nst) load((i + 3) * kR, s1);
    mma(1);
    if (i + 2 < nst) store(s0, 0);
    __syncthreads();
  }
  const float sa = w.s[a];
  uint16_t *out = g.out + (int64_t)a * r * C;
  float *part = g.part + (int64_t)blockIdx.y * r * C;
#pragma unroll
  for (int t = 0; t < TJ; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // 4 ranks from j of column c, or rank j of 4 columns from c
      const int j = t * 16 + (g.transposed ? 4 * g16 : l16);
      const int64_t c = c0 + wave * 32 + u * 16 + (g.transposed ? l16 : 4 * g16);
      if (j >= r || c >= C) continue;
      const int64_t at = g.transposed ? c * r + j : j * C + c;
      const f32x4 y = acc[t][u];
      const uint2 z = me ? make_uint2(pack_bf16x2(sa * y[0], sa * y[1]), pack_bf16x2(sa * y[2], sa * y[3]))
                         : make_uint2(0, 0);
      if (g.transposed && (r & 3) != 0) {   // rows of out that are not 8-byte aligned
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (j + v >= r) break;
          if (nb > 1)
            part[at + v] = y[v];
          else
            out[at + v] = (uint16_t)((v < 2 ? z.x : z.y) >> (16 * (v & 1)));
        }
      } else if (nb > 1) {
        *reinterpret_cast<f32x4 *>(part + at) = y;
      } else {
        *reinterpret_cast<uint2 *>(out + at) = z;
      }
    }
}

// out[a] = bf16(s[a] * (sum over the adapter's blocks of part)) where the adapter (blockIdx.y) has more
// than one block, zeros where it has none; n values an adapter, two a thread (n is even: r C with
// C % 8 == 0).
__global__ void multi_sum_final_kernel(SumArgs w, MultiPlan pl) {
  const MultiSum g = blockIdx.z ? w.g[1] : w.g[0];
  const int32_t *first = pl.table[kPlanSum];
  const int a = blockIdx.y, lo = first[a], nb = first[a + 1] - lo;
  const int64_t n = (int64_t)w.r * g.c;
  if (nb == 1) return;
  const float sa = w.s[a];
  for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) * 2; i < n; i += (int64_t)gridDim.x * blockDim.x * 2) {
    const float *pa = g.part + (int64_t)lo * n + i;
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
    *reinterpret_cast<uint32_t *>(g.out + a * n + i) = nb ? pack_bf16x2(sa * x[0], sa * x[1]) : 0u;
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

hipError_t launch_multi_plan(const int32_t *ids, int64_t M, int L, const MultiPlan &pl, const MultiPad &pd,
                             const MultiFactors &f, hipStream_t st) {
  if (L < 1 || L > kMultiMaxAdapters || M < 1 || M >= (int64_t(1) << 30)) return hipErrorInvalidValue;
  PlanWork w{};
  w.pad = PadArgs{pd.src, pd.dst, pd.src ? pd.rows : 0, pd.r, pd.rp};
  const int64_t pads = (w.pad.rows * pd.rp + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  w.pad_blocks = (int)(pads < 1024 ? pads : 1024);
  if (f.Bt) {
    if (f.rp < f.r || (f.rp & 7) != 0 || (f.n & 7) != 0) return hipErrorInvalidValue;
    const int lr = rank_log(f.r);
    w.tr[0] = TransposeArgs{f.B, f.Bt, f.n, f.r, f.n, 12 - lr, lr};
    if (f.At) w.tr[1] = TransposeArgs{f.A, f.At, f.r, f.k, f.rp, lr, 12 - lr};
  }
  const int64_t blocks = 1 + w.pad_blocks + (w.tr[0].blocks() + w.tr[1].blocks()) * L;
  if (blocks >= (int64_t(1) << 32) / kPlanThreads) return hipErrorInvalidValue;
  const size_t lds = sizeof(int32_t) * kPlanWaves * (L + 1);
  multi_plan_kernel<<<dim3((unsigned)blocks), dim3(kPlanThreads), lds, st>>>(ids, M, L, pl, w);
  return hipGetLastError();
}

// Rows per block of the row projection: 16 up to 1024 rows, where the groups of a serving batch are a
// few rows each, else 64, which reads an adapter's factor a fourth as often.
static int multi_rows_block(int64_t M) { return M <= 1024 ? 16 : 64; }

// Splits of its reduction, at least 256 elements each: the workgroups of all blocks (an adapter's last one is
// half full on average) stay under the 1024 that fit on the card at once with rank 64. Just above it, 8192 rows
// of 4 adapters and rank 64, forward and backward, took 1568 us instead of 1548.
int multi_rows_splits(int64_t M, int64_t Lr, int L) {
  const int64_t wgs = (M + multi_rows_block(M) - 1) / multi_rows_block(M) + (L + 1) / 2;
  const int64_t s = std::min(int64_t(1000) / wgs, (Lr + 255) / 256);
  return (int)std::max(s, int64_t(1));
}

hipError_t launch_multi_rows(const MultiRows *g, int count, int64_t M, int r, int rp, int L, const MultiPlan &pl,
                             hipStream_t st) {
  if (count < 1 || count > 2 || rp < r || (rp & 7) != 0) return hipErrorInvalidValue;
  const int64_t rows = multi_rows_block(M);
  RowsArgs w{{g[0], g[count - 1]}, {}, M, r, rp, L};
  int most = 1;
  for (int i = 0; i < 2; ++i) {
    if ((w.g[i].l & 7) != 0 || w.g[i].splits < 1 || w.g[i].splits > 65535) return hipErrorInvalidValue;
    w.lsplit[i] = ((w.g[i].l + w.g[i].splits - 1) / w.g[i].splits + 63) / 64 * 64;
    most = most > w.g[i].splits ? most : w.g[i].splits;
  }
  int64_t blocks = (M + (rows - 1) * (L + 1)) / rows;   // >= the sum of ceil(rows of a group / rows)
  blocks = blocks < M ? blocks : M;
  const dim3 grid((unsigned)blocks, (unsigned)most, (unsigned)count);
  switch ((r + 15) / 16) {
#define MR_CASE(T)                                                       \
  case T:                                                                \
    if (rows == 16)                                                      \
      multi_rows16_kernel<T><<<grid, dim3(256), 0, st>>>(w, pl);         \
    else                                                                 \
      multi_rows64_kernel<T><<<grid, dim3(256), 0, st>>>(w, pl);         \
    break;
    MR_CASE(1) MR_CASE(2) MR_CASE(3) MR_CASE(4) MR_CASE(5) MR_CASE(6) MR_CASE(7) MR_CASE(8)
#undef MR_CASE
    default: return hipErrorInvalidValue;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!g[0].out && !g[0].padded && !g[0].wide)) return e;
  multi_rows_sum_kernel<<<dim3((unsigned)blocks_for(M * rp), (unsigned)count), dim3(256), 0, st>>>(w);
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
// tiles of both sums, 64 to 1024 rows. Up to kMultiSmallM rows are one block.
int multi_sum_rows(int64_t M, int64_t c0, int64_t c1) {
  if (M <= kMultiSmallM) return kMultiSmallM;
  const int64_t tiles = (c0 + kCB - 1) / kCB + (c1 + kCB - 1) / kCB;
  const int64_t rows = (M * tiles / 1024 + kRB - 1) / kRB * kRB;
  return (int)(rows < kRB ? kRB : rows < kSumRows ? rows : kSumRows);
}
int64_t multi_sum_blocks(int64_t M, int64_t c0, int64_t c1, int L) {
  if (M <= kMultiSmallM) return 0;   // nothing to add afterwards
  const int64_t rows = multi_sum_rows(M, c0, c1), b = (M + (rows - 1) * L) / rows;   // >= the sum of ceil(rows of a / rows)
  return b < M ? b : M;
}

hipError_t launch_multi_sums(const MultiSum &a, const MultiSum &b, int64_t M, int r, int rp, int L, const float *s,
                             const MultiPlan &pl, hipStream_t st) {
  const SumArgs w{{a, b}, s, r, rp, L};
  // Stages of 32 rows let more of the workgroups of many adapters with few rows share a CU (forward and
  // backward of 255 rows of 60 adapters, 4096 x 4096: 125 -> 111 us); an adapter of many rows then takes twice
  // the steps (250 rows of one: 100 -> 108 us).
  const bool small = M <= kMultiSmallM, few = small && M <= 32 * (int64_t)L;
  const int64_t most = std::max(a.c, b.c), tiles = (most + kCB - 1) / kCB;
  const int64_t blocks = small ? L : multi_sum_blocks(M, a.c, b.c, L);
  if (rp < r || (rp & 7) != 0 || ((a.c | b.c) & 7) != 0 || pl.rows[kPlanSum] != multi_sum_rows(M, a.c, b.c) ||
      blocks > 65535)
    return hipErrorInvalidValue;
  const dim3 grid((unsigned)tiles, (unsigned)blocks, 2);
  switch ((r + 15) / 16) {
#define MS_CASE(T)                                                       \
  case T:                                                                \
    if (few)                                                             \
      multi_sum_kernel<T, true, 32><<<grid, dim3(256), 0, st>>>(w, pl);  \
    else if (small)                                                      \
      multi_sum_kernel<T, true, kRB><<<grid, dim3(256), 0, st>>>(w, pl); \
    else                                                                 \
      multi_sum_kernel<T, false, kRB><<<grid, dim3(256), 0, st>>>(w, pl);\
    break;
    MS_CASE(1) MS_CASE(2) MS_CASE(3) MS_CASE(4) MS_CASE(5) MS_CASE(6) MS_CASE(7) MS_CASE(8)
#undef MS_CASE
    default: return hipErrorInvalidValue;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || small) return e;
  const int64_t x = std::min<int64_t>(((int64_t)r * most / 2 + 255) / 256, 1024);
  multi_sum_final_kernel<<<dim3((unsigned)x, (unsigned)L, 2), dim3(256), 0, st>>>(w, pl);
  return hipGetLastError();
}

hipError_t launch_multi_pad(const uint16_t *src, int64_t rows, int r, int rp, uint16_t *dst, hipStream_t st) {
  const PadArgs p{src, dst, rows, r, rp};
  multi_pad_kernel<<<dim3((unsigned)blocks_for(rows * rp)), dim3(256), 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace nf4q
