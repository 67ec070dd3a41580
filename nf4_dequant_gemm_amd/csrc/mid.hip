// Forward of the layer with an adapter of its own for every row, for the batches between one row and a
// full grid of 256 x 256 tiles: Y = X deq(W)^T + s_a T B_a^T (gfx950).
//
// At these sizes the large kernel has too few tiles for the 256 CUs and the 16-row stream kernel takes
// too few rows. A workgroup of 8 waves takes 16 kMT rows and 32 kNW columns: kNW waves side by side,
// each 32 columns, times kKW = 8 / kNW waves that take turns along K, in steps of kBlk blocks of 64.
//   * Weight codes go straight to the registers of the lanes that multiply them: lane (g, l) of a
//     16-row tile loads 16 bytes of row l for each 128 elements (whole 64-byte runs of a row), and two
//     v_permlane32_swap hand every lane 8 bytes of each of the two blocks, so that an MFMA sees one
//     block only.
//   * NF4: a code byte (two elements) becomes a pair of unscaled bf16 levels (rounded: the matrix
//     instructions take bf16; the layer's kernels round level times constant) by one lookup in a
//     256-entry LDS table held 64 times (entry e of copy c at byte 256 e + 4 c: a byte permute forms
//     the address, every lane has its own bank); the block constant scales the block's float32 sum.
//     That is one vector instruction and one LDS read for two elements, where decoding through a table
//     of scaled values in registers takes nine: the 16-row launch of a 4096 x 4096 weight took 33 us
//     that way.
//   * E2M1: a lane's 8 bytes are one group of 16. The values times the group scale are exact in bf16;
//     the tensor scale multiplies the sums at the end.
//   * X goes to LDS by DMA, 16-byte chunk c of a row's 256 bytes (128 elements) at slot c ^ (row % 16),
//     which gives the 16 rows of an operand read distinct slots of the 256-byte bank window.
//   * Codes, constants and X of the next two steps are in flight during a step; one barrier per step.
// The kKW sums of a tile meet in LDS, in wave order, which also turns them round for whole row pieces.
// With few tiles the reduction is also split over workgroups. All write float32 sums, which
// mid_final_kernel adds in order; it then applies the low-rank term and writes Y and T.
//
// T of at most 256 rows is formed in the same launch, by workgroups of their own that each take 1024
// elements of the reduction for 16 rows of an adapter (multi_rows_of) and write float32 sums too: a
// launch for T alone took 6 to 9 us, and nothing needs T before the end. They come last in the grid, for
// the CUs that the tiles leave idle. More rows bring T's sums from the row projection.
//
// What bounds it: a step's matrix (37% of the time at 7 row tiles) and vector instructions (34%: two of
// the three for each product scale and add a block's sums) take turns on a SIMD, and its LDS reads (40% of
// the LDS's time) do not hide behind them completely. 200 rows x 4096 x 11008: 43 us, and 10 us for the
// last launch; 1111 rows x 2880 x 2952 in E2M1: 36 and 16 us; one row x 4096 x 4096: 8.3 and 3.9 us.
#include "common.h"
#include "launch.h"
#include "multi.h"

namespace nf4q {
namespace {

constexpr int kThreads = 512;

struct MidArgs {
  const uint16_t *X;
  WDesc w;
  int64_t M, N, K;
  uint16_t *Y;         // [M][N]
  float *part;         // [splits][M][N]
  int splits;
  Tables t;
  // T's sums, [tsplits][M][mu.r] (tsplits 0: T is whole, in mu.P), and T [M][ra], written by
  // mid_final_kernel; mu.r is the rank ra padded to a multiple of 8
  float *tpart;
  int tsplits, ra;
  uint16_t *T;
  // T formed in the launch: the workgroups from tfirst on, from A [L][ra][K], and the last of them puts
  // the rows in the order of their adapters: order [M]
  int tfirst;
  const uint16_t *A;
  int32_t *order;
};
constexpr int kTSlice = 1024;   // reduction elements of a workgroup that forms T

// Y columns n .. n + 3 of row m from float32 sums.
__device__ __forceinline__ void store4(uint16_t *Y, int64_t N, int64_t m, int64_t n, const f32x4 &a) {
  *reinterpret_cast<uint2 *>(Y + m * N + n) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
}

// The tensor scale of an E2M1 weight (1 for an all-zero weight, whose group scales are all 0).
__device__ __forceinline__ float tensor_scale(const WDesc &w) {
  const float S = *w.scale;
  return S > 0.f ? S : 1.f;
}

struct Pair {
  uint32_t a, b;
};
// (a, b) -> a's lower 32 lanes with b's lower 32 lanes above them, a's upper with b's upper above.
__device__ __forceinline__ Pair swap_halves(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return Pair{r[0], r[1]};
}

// kFmt: 0 NF4 with float32 constants, 1 NF4 double-quantised, 2 E2M1. kMT: row tiles of 16. kBlk: blocks
// of a wave's step (2 or 4). kAl: K is a multiple of 64 kBlk, so that a row's constants of a step are
// one aligned piece (double-quantised: with one run scale); otherwise they are loaded one by one and
// the last step may hold blocks past K, whose X reads as zero.
template <int kFmt, int kMT, int kNW, int kBlk, bool kAl>
__global__ __launch_bounds__(kThreads) void mid_kernel(MidArgs g, MultiArgs mu) {
  constexpr bool kDQ = kFmt == 1, kFP4 = kFmt == 2;
  constexpr int kKW = 8 / kNW, kH = kBlk / 2;       // 128-element halves of a step
  constexpr int kMX = kBlk == 2 ? (kMT + 1) / 2 * 2 : kMT;   // row tiles of X copied: whole pieces for 8 waves
  constexpr int kHalf = kMX * 16 * 16;              // 16-byte chunks of one half's X
  constexpr int kSlice = kH * kHalf;                // of one wave step's
  constexpr int kPieces = kKW * kSlice / 64;        // 1 KB DMA pieces per step
  static_assert(kPieces % 8 == 0, "every wave issues the same copies");
  // Vector-memory operations a wave issues per step: its copies, the codes and the constants. The wait
  // at the start of a step leaves those of the step after it in flight.
  constexpr int kStepLoads =
      kPieces / 8 + 2 * (kH + (kAl ? (kDQ ? 2 : 1) : kBlk * (kDQ ? 2 : 1)));
  // separate arrays, so that the compiler does not take reads of one for reads of a copy in flight
  __shared__ uint4 sX0[kKW * kSlice], sX1[kKW * kSlice], sX2[kKW * kSlice];
  // the level table; at the end the sums of a row tile: [wave][row][32 columns, padded to 36]
  constexpr int kPad = 36, kTiles = kKW == 1 ? 1 : kMT;   // row tiles in LDS at a time
  constexpr int kSums = 8 * kTiles * 16 * kPad, kTab = kFP4 ? 0 : 256 * 64;
  __shared__ __align__(16) uint32_t stab[kSums > kTab ? kSums : kTab];
  const int block = blockIdx.x;
  if (block >= g.tfirst) {
    static_assert(kMultiSmallT<8, 2> <= sizeof(stab), "T's sums fit the table");
    const int nj = (mu.r + 31) / 32;
    const int tb = block - g.tfirst;
    if (tb == (int)g.M * nj * g.tsplits) {   // a row's place: the rows before it by adapter, then by number
      int *key = reinterpret_cast<int *>(stab);
      const int i = threadIdx.x, M = (int)g.M;
      int mine = 0;
      if (i < M) {
        const int a = mu.ids[i];
        key[i] = mine = a >= 0 && a < mu.L ? a : mu.L;
      }
      __syncthreads();
      if (i < M) {
        int at = 0;
        for (int j = 0; j < M; ++j) at += key[j] < mine || (key[j] == mine && j < i);
        g.order[at] = i;
      }
      return;
    }
    const int ts = tb % g.tsplits, j = tb / g.tsplits % nj, row = tb / g.tsplits / nj;
    const int64_t le = (int64_t)(ts + 1) * kTSlice;
    float *tp = g.tpart + (int64_t)ts * g.M * mu.r;
    multi_rows_of<8, 2, 4>(g.X, g.K, g.A, (int64_t)g.ra * g.K, g.K, mu.ids, (int)g.M, (int64_t)ts * kTSlice,
                           le < g.K ? le : g.K, g.ra, mu.r, mu.L, row, j * 32, stab,
                           [&](int i, int jj, float s) { tp[(int64_t)i * mu.r + jj] = s; });
    return;
  }
  const int cols = (int)((g.N + 32 * kNW - 1) / (32 * kNW)), rowb = (int)((g.M + 16 * kMT - 1) / (16 * kMT));
  const int bx = block % cols, by = block / cols % rowb, bz = block / cols / rowb;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nw = wave % kNW, kw = wave / kNW;
  const int g16 = lane >> 4, l16 = lane & 15;
  const int64_t K = g.K, N = g.N;
  const int kblk = (int)(K / 64);
  const int64_t n0 = (int64_t)bx * 32 * kNW + 32 * nw;   // this wave's columns
  const int64_t m0 = (int64_t)by * 16 * kMT;
  const int64_t rows_m = g.M - m0 < 16 * kMT ? g.M - m0 : 16 * kMT;
  const int64_t rows_n = n0 >= N ? 0 : N - n0 < 32 ? N - n0 : 32;
  const int64_t nb = n0 < N ? n0 : 0;               // a wave past the last column reads nothing
  // this workgroup's steps [sbeg, send); wave kw takes sbeg + kw, + kKW, ...
  const int nsteps = (kblk + kBlk - 1) / kBlk;
  const int sbeg = (int)((int64_t)bz * nsteps / g.splits);
  const int send = (int)((int64_t)(bz + 1) * nsteps / g.splits);
  const int iters = (send - sbeg + kKW - 1) / kKW;
  constexpr uint32_t kNone = 0x80000000u;           // an offset outside every buffer: reads zero

  const __amdgpu_buffer_rsrc_t rX = make_rsrc(g.X + m0 * K, rows_m * K * 2);
  const __amdgpu_buffer_rsrc_t rC = make_rsrc(g.w.codes + nb * (K / 2), rows_n * (K / 2));
  const __amdgpu_buffer_rsrc_t rQ =
      kFP4  ? make_rsrc(reinterpret_cast<const uint8_t *>(g.w.absmax) + nb * (K / 16), rows_n * (K / 16))
      : kDQ ? make_rsrc(reinterpret_cast<const int8_t *>(g.w.absmax) + nb * kblk, rows_n * kblk)
            : make_rsrc(reinterpret_cast<const float *>(g.w.absmax) + nb * kblk, rows_n * kblk * 4);
  const int64_t nruns = (g.w.n * kblk + 255) / 256;
  const __amdgpu_buffer_rsrc_t rS = make_rsrc(g.w.scale, kDQ ? nruns * 4 : 0);

  // X pieces of 1 KB: four rows of one half; lane L writes LDS chunk L % 16 of row 4 q + L / 16, which
  // holds the row's chunk (L % 16) ^ (row % 16).
  auto dma_x = [&](int it, uint4 *dst) {
#pragma unroll
    for (int i = 0; i < kPieces / 8; ++i) {
      const int p = wave + 8 * i;
      const int half = p / (4 * kMX), q = p % (4 * kMX);   // half of the kKW kH of this step
      const int row = 4 * q + (lane >> 4);
      const int chunk = (lane & 15) ^ (row & 15);
      const int st = sbeg + it * kKW + half / kH;
      const int k = (st * kH + half % kH) * 128 + chunk * 8;
      // rows past M, steps past the end and chunks past K read as zero (the last by arithmetic: as a
      // condition it made the compiler spill 200 registers)
      uint32_t off = st < send ? (uint32_t)((row * K + k) * 2) : kNone;
      if (!kAl) off |= (uint32_t)(((int)K - 1 - k) >> 31) & kNone;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rX, (__attribute__((address_space(3))) void *)(dst + p * 64), 16, off,
                                               0, 0, 0);
    }
  };
  struct Codes {
    u32x4 c[2][kH];
    uint32_t q[2][kBlk];   // NF4: int8 code or float bits of each block; E2M1: its four group scales
    uint32_t s[2][kAl ? 1 : kBlk];
  };
  // byte of the lane's codes and first block of its row, in the wave's rows (and, for the run scales, in
  // the weight: blocks fit 32 bits)
  uint32_t cbase[2], bbase[2];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    cbase[nt] = (uint32_t)((nt * 16 + l16) * (K / 2) + 16 * g16);
    bbase[nt] = (uint32_t)((nt * 16 + l16) * kblk);
  }
  const uint32_t wblk = (uint32_t)(nb * kblk);
  auto load_c = [&](int it, Codes &c) {
    const int st = sbeg + it * kKW + kw;
    const bool in = st < send;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
      for (int h = 0; h < kH; ++h)
        c.c[nt][h] = __builtin_amdgcn_raw_buffer_load_b128(
            rC, in ? cbase[nt] + (st * kH + h) * 64 : kNone, 0, 0);
      const uint32_t b0 = bbase[nt] + st * kBlk;
      if constexpr (kAl) {
        if constexpr (kDQ) {
          c.q[nt][0] = kBlk == 4 ? __builtin_amdgcn_raw_buffer_load_b32(rQ, in ? b0 : kNone, 0, 0)
                                 : __builtin_amdgcn_raw_buffer_load_b16(rQ, in ? b0 : kNone, 0, 0);
          // a step past the end: nothing of the next row's run, as below
          c.s[nt][0] = __builtin_amdgcn_raw_buffer_load_b32(rS, in ? ((wblk + b0) >> 8) * 4 : kNone, 0, 0);
        } else if constexpr (kBlk == 4) {
          const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rQ, in ? b0 * 4 : kNone, 0, 0);
#pragma unroll
          for (int b = 0; b < 4; ++b) c.q[nt][b] = v[b];
        } else {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rQ, in ? b0 * 4 : kNone, 0, 0);
          c.q[nt][0] = v[0];
          c.q[nt][1] = v[1];
        }
      } else {
#pragma unroll
        for (int b = 0; b < kBlk; ++b) {
          // a block past K: a constant of 0, not the next row's, whose Inf or NaN would meet the zeros of X
          // (by arithmetic, as the copies of X)
          const uint32_t past = (uint32_t)((kblk - 1 - st * kBlk - b) >> 31) & kNone;
          if constexpr (kDQ) {
            c.q[nt][b] = __builtin_amdgcn_raw_buffer_load_b8(rQ, (in ? b0 + b : kNone) | past, 0, 0);
            c.s[nt][b] = __builtin_amdgcn_raw_buffer_load_b32(rS, (((wblk + b0 + b) >> 8) * 4) | past, 0, 0);
          } else {
            c.q[nt][b] = __builtin_amdgcn_raw_buffer_load_b32(rQ, (in ? (b0 + b) * 4 : kNone) | past, 0, 0);
          }
        }
      }
    }
  };

  f32x4 acc[2][kMT];   // lane (g16, l16): rows 16 mt + 4 g16 + v of column 16 nt + l16
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) acc[nt][mt] = f32x4{0.f, 0.f, 0.f, 0.f};

  const uint32_t copy = (uint32_t)lane * 4;
  const char *tab = reinterpret_cast<const char *>(stab);
  // after the swap lane group g holds elements 16 sg .. 16 sg + 15 of a block, sg = 0, 2, 1, 3
  const int sg = ((g16 & 1) << 1) | (g16 >> 1);

  // A block's weights as operands, decoded in four parts (column tile, half), and its constants.
  struct Block {
    bf16x8 w[2][2];
    float a[2];   // NF4: the block's constant; E2M1: the lane's group scale
  };
  Pair turned[2][2];   // the lane's 8 bytes of a half's first and second block
  auto decode = [&](const Codes &c, int blk, int part, Block &d) {
    const int nt = part >> 1, e = part & 1, h = blk >> 1;
    if ((blk & 1) == 0) turned[nt][e] = swap_halves(c.c[nt][h][e], c.c[nt][h][e + 2]);
    const uint32_t code = blk & 1 ? turned[nt][e].b : turned[nt][e].a;
    if constexpr (kFP4) {
      if (e == 0) d.a[nt] = __builtin_amdgcn_cvt_f32_fp8((int)(c.q[nt][blk] >> (8 * sg)), 0);
      const float s = d.a[nt];
      // bytes hold the earlier element in the high nibble
      const uint32_t u = ((code >> 4) & 0x0F0F0F0Fu) | ((code << 4) & 0xF0F0F0F0u);
      const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 0);
      const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 1);
      const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 2);
      const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 3);
      d.w[nt][e] = __builtin_bit_cast(
          bf16x8, make_uint4(pack_bf16x2(p0[0] * s, p0[1] * s), pack_bf16x2(p1[0] * s, p1[1] * s),
                             pack_bf16x2(p2[0] * s, p2[1] * s), pack_bf16x2(p3[0] * s, p3[1] * s)));
    } else {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = perm(code, copy, 0x0C0C0400u | ((4u + i) << 8));
        o[i] = *reinterpret_cast<const uint32_t *>(tab + at);
      }
      d.w[nt][e] = __builtin_bit_cast(bf16x8, make_uint4(o[0], o[1], o[2], o[3]));
      if (e == 0) {
        if constexpr (kDQ)
          d.a[nt] = int8_code(kAl ? c.q[nt][0] >> (8 * blk) : c.q[nt][blk]) * __uint_as_float(c.s[nt][kAl ? 0 : blk]);
        else
          d.a[nt] = __uint_as_float(c.q[nt][blk]);
      }
    }
  };

  // One step's blocks, a row tile at a time, in an order that keeps the LDS reads behind the products:
  // while a row tile multiplies, the next one's X and a part of the next block's weights are read, and
  // the tile before is scaled and added.
  auto compute = [&](const Codes &c, const uint4 *sX) {
    const uint4 *mine = sX + kw * kSlice;
    constexpr int kAll = kBlk * kMT;
    Block d[2];
    bf16x8 x[2][2];
    f32x4 part[2][2];
    float scale[2][2];
    auto load_x = [&](int i) {
      const int blk = i / kMT, mt = i % kMT;
      const uint4 *row = mine + (blk >> 1) * kHalf + (mt * 16 + l16) * 16;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        x[i & 1][e] = __builtin_bit_cast(bf16x8, row[(8 * (blk & 1) + 2 * sg + e) ^ l16]);
    };
    auto add = [&](int i) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[nt][i % kMT][v] += scale[i & 1][nt] * part[i & 1][nt][v];
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) decode(c, 0, q, d[0]);
    load_x(0);
#pragma unroll
    for (int i = 0; i < kAll; ++i) {
      const int blk = i / kMT, mt = i % kMT;
      const Block &now = d[blk & 1];
      if (i + 1 < kAll) load_x(i + 1);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        scale[i & 1][nt] = now.a[nt];
        if constexpr (kFP4)
          acc[nt][mt] = mfma16x16x32(x[i & 1][0], now.w[nt][0], acc[nt][mt]);
        else
          part[i & 1][nt] = mfma16x16x32(x[i & 1][0], now.w[nt][0], f32x4{0.f, 0.f, 0.f, 0.f});
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        f32x4 &to = kFP4 ? acc[nt][mt] : part[i & 1][nt];
        to = mfma16x16x32(x[i & 1][1], now.w[nt][1], to);
      }
      if (!kFP4 && i > 0) add(i - 1);
      if (blk + 1 < kBlk) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q * kMT / 4 == mt) decode(c, blk + 1, q, d[(blk + 1) & 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!kFP4) add(kAll - 1);
  };

  // Step it: wait for its X and codes (requested two steps ago; those of the next step stay in flight),
  // barrier (everyone's copies have landed and everyone is done with the step before, whose buffer
  // takes the next copies), request step it + 2, multiply.
  Codes c0, c1, c2;
  auto step = [&](int it, uint4 *cur, uint4 *next, Codes &c, Codes &cn) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kStepLoads) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    dma_x(it + 2, next);   // past the last step: zeros, into a buffer nobody reads any more
    load_c(it + 2, cn);
    __builtin_amdgcn_sched_barrier(0);   // the decode of this step stays behind the requests
    compute(c, cur);
    __builtin_amdgcn_sched_barrier(0);
  };
  dma_x(0, sX0);
  load_c(0, c0);
  __builtin_amdgcn_sched_barrier(0);
  dma_x(1, sX1);
  load_c(1, c1);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (!kFP4) {   // uint4 i of the table: four copies of entry i / 16
    float *lv = reinterpret_cast<float *>(sX2);   // its first copy is requested after the first barrier
    if (tid == 0) {
#pragma unroll
      for (int j = 0; j < 16; ++j) lv[j] = g.t.level[j];
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    for (int i = tid; i < 256 * 16; i += kThreads) {
      const uint32_t v = pack_bf16x2(lv[i >> 8], lv[(i >> 4) & 15]);
      reinterpret_cast<uint4 *>(stab)[i] = make_uint4(v, v, v, v);
    }
  }
  int it = 0;
#pragma unroll 1
  for (; it + 3 <= iters; it += 3) {
    step(it, sX0, sX2, c0, c2);
    step(it + 1, sX1, sX0, c1, c0);
    step(it + 2, sX2, sX1, c2, c1);
  }
  if (it < iters) step(it, sX0, sX2, c0, c2);
  if (it + 1 < iters) step(it + 1, sX1, sX0, c1, c0);
  // the copies of the steps past the end have landed, and everyone is done with the table
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // Wave (nw, kw) adds the kKW sums of its columns for row tiles kw, kw + kKW, ... and reads 4 columns
  // of a row at a time.
  float *sums = reinterpret_cast<float *>(stab);
  auto park = [&](int mt) {
    float *p = sums + ((wave * kTiles + mt % kTiles) * 16 + 4 * g16) * kPad + l16;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int v = 0; v < 4; ++v) p[v * kPad + 16 * nt] = acc[nt][mt][v];
  };
  const float tsc = kFP4 ? tensor_scale(g.w) : 1.f;
  auto finish = [&](int mt) {
    f32x4 y[2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      auto at = [&](int k) {
        return *reinterpret_cast<const f32x4 *>(
            sums + (((k * kNW + nw) * kTiles + mt % kTiles) * 16 + l16) * kPad + 16 * nt + 4 * g16);
      };
      y[nt] = at(kKW == 1 ? kw : 0);
#pragma unroll
      for (int k = 1; k < kKW; ++k) y[nt] += at(k);
      if (kFP4) y[nt] *= tsc;
    }
    const int64_t m = m0 + mt * 16 + l16;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int64_t n = n0 + nt * 16 + 4 * g16;
      if (m < g.M && n < N) *reinterpret_cast<f32x4 *>(g.part + ((int64_t)bz * g.M + m) * N + n) = y[nt];
    }
  };
  if constexpr (kKW == 1) {   // a wave's own tile: its LDS accesses are in order
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      park(mt);
      __builtin_amdgcn_wave_barrier();
      finish(mt);
      __builtin_amdgcn_wave_barrier();
    }
  } else {
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) park(mt);
    __syncthreads();
#pragma unroll 1
    for (int mt = kw; mt < kMT; mt += kKW) finish(mt);
  }
}

// Y (or dX) from the float32 sums of the launch before, added in order, and the low-rank term, with T from
// its own sums (written here, by the workgroups of the first columns) or T (U) from memory. One wave:
// 16 rows, in the order of their adapters (perm, unless there is one row tile only), and kFinalTiles
// 16-column tiles. It is bound by its chain of loads, so those of the first splits are in flight
// during the term. 200 rows of 64 adapters x 11008, two splits: 10.4 us for 22 MB and the factors; 14.4 us
// with the rows in the batch's order (14 adapters to a row tile instead of 5).
template <int kFinalTiles>
__global__ __launch_bounds__(64) void mid_final_kernel(MidArgs g, MultiArgs mu) {
  // splits and adapters whose loads are in flight together: fewer with 64 columns, where there are waves
  // enough to hide them if the registers let them on (1000 rows x 8000, whole call, 119 -> 115 us)
  constexpr int kAhead = kFinalTiles == 2 ? 4 : 2, kTogether = kAhead;
  const int lane = threadIdx.x, g16 = lane >> 4, l16 = lane & 15;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * kFinalTiles;
  int64_t m = (int64_t)blockIdx.y * 16 + l16;
  const bool have = m < g.M;
  if (mu.perm) m = have ? mu.perm[m] : 0;
  int id = have ? mu.ids[m] : -1;
  id = id >= 0 && id < mu.L ? id : -1;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  auto load = [&](int s0, f32x4 (&v)[kAhead][kFinalTiles]) {   // kAhead splits
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int nt = 0; nt < kFinalTiles; ++nt) {
        const int64_t n = n0 + nt * 16 + 4 * g16;
        v[s][nt] = s0 + s < g.splits && have && n < g.N
                       ? *reinterpret_cast<const f32x4 *>(g.part + ((int64_t)(s0 + s) * g.M + m) * g.N + n)
                       : zero;
      }
  };
  f32x4 v[kAhead][kFinalTiles], y[kFinalTiles], term[kFinalTiles];
  load(0, v);
#pragma unroll
  for (int nt = 0; nt < kFinalTiles; ++nt) y[nt] = term[nt] = zero;
  multi_term_rows<kTogether>(term, mu, id, n0, g.N, [&](int j) {
    const bool mine = have && j < mu.r;
    if (!g.tsplits)
      return __builtin_bit_cast(bf16x8, mine ? *reinterpret_cast<const u32x4 *>(mu.P + m * mu.r + j)
                                             : u32x4{0u, 0u, 0u, 0u});
    f32x4 a = zero, b = zero;
    const float *tp = g.tpart + m * mu.r + j;
    for (int t0 = 0; t0 < g.tsplits; t0 += 4) {
      f32x4 x[4][2];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[t][h] = mine && t0 + t < g.tsplits
                        ? *reinterpret_cast<const f32x4 *>(tp + (t0 + t) * g.M * mu.r + 4 * h) : zero;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        a += x[t][0];
        b += x[t][1];
      }
    }
    if (mine && blockIdx.x == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < g.ra) g.T[m * g.ra + j + e] = (uint16_t)(pack_bf16x2(e < 4 ? a[e & 3] : b[e & 3], 0.f) & 0xFFFFu);
    }
    return __builtin_bit_cast(bf16x8, make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                 pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])));
  });
  for (int s0 = 0;;) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int nt = 0; nt < kFinalTiles; ++nt) y[nt] += v[s][nt];
    s0 += kAhead;
    if (s0 >= g.splits) break;
    load(s0, v);
  }
#pragma unroll
  for (int nt = 0; nt < kFinalTiles; ++nt) {
    const int64_t n = n0 + nt * 16 + 4 * g16;
    if (have && n < g.N) store4(g.Y, g.N, m, n, y[nt] + term[nt]);
  }
}

// 64 columns a wave read a row tile's adapters least often; a grid of under 8 such waves for each CU is
// latency alone, and 32 columns then shorten every wave (4096 columns: 12 rows 17.4 -> 15.7 us for the
// whole call; 500 rows, 64 adapters 61.0 -> 64.5 us, where there are enough waves without).
void launch_final(const MidArgs &a, const MultiArgs &mu, hipStream_t st) {
  const int64_t rows = (a.M + 15) / 16, cols = (a.N + 63) / 64;
  if (rows * cols < 8 * 256)
    mid_final_kernel<2><<<dim3((unsigned)((a.N + 31) / 32), (unsigned)rows), dim3(64), 0, st>>>(a, mu);
  else
    mid_final_kernel<4><<<dim3((unsigned)cols, (unsigned)rows), dim3(64), 0, st>>>(a, mu);
}

template <int kMT, int kNW, int kBlk, bool kAl>
void launch_fmt(const MidArgs &a, const MultiArgs &mu, unsigned grid, hipStream_t st) {
  if (a.w.fp4)
    mid_kernel<2, kMT, kNW, kBlk, kAl><<<dim3(grid), dim3(kThreads), 0, st>>>(a, mu);
  else if (a.w.dq)
    mid_kernel<1, kMT, kNW, kBlk, kAl><<<dim3(grid), dim3(kThreads), 0, st>>>(a, mu);
  else
    mid_kernel<0, kMT, kNW, kBlk, kAl><<<dim3(grid), dim3(kThreads), 0, st>>>(a, mu);
}

// The split of a launch: rows of a workgroup (up to 8 row tiles of 16), waves side by side, blocks of a
// step (what the LDS holds three times beside the table) and splits of the reduction. Of all of them the
// least of (rounds of 256 workgroups) x (start and end of one, and its steps) plus the traffic of the
// float32 sums, in us, with the times measured for 16 to 128 rows. With one row tile T's workgroups
// count as well: in a second round they made 1 to 12 rows x 4096 x 4096 1.1 to 1.6 us slower (with
// more rows most of them have no row to start from, and a few idle CUs are enough: where there are none
// 128 rows x 8192 x 4096 took 40.6 us instead of 37.7).
struct MidShape {
  int mt, nw, blk, splits;
  bool al;
};
MidShape mid_shape(int64_t M, int64_t N, int64_t K) {
  MidShape best{};
  const int64_t t = (M + 15) / 16, for_t = M <= 16 ? M * ((K + kTSlice - 1) / kTSlice) : 0;
  double least = 0;
  for (int mt = 1; mt <= 8 && mt <= t; ++mt) {
    const int64_t row_blocks = (t + mt - 1) / mt;
    MidShape s{mt, mt <= 2 ? 4 : 8, mt <= 4 ? 4 : 2, 1, false};
    s.al = K % (64 * s.blk) == 0;
    const int64_t kw = 8 / s.nw, wgs = row_blocks * ((N + 32 * s.nw - 1) / (32 * s.nw));
    const int64_t steps = (K / 64 + s.blk - 1) / s.blk;
    const double per_step = s.blk * (0.3 + 0.13 * mt);
    for (int64_t sp = 1; sp == 1 || (sp <= 16 && sp * kw <= steps); ++sp) {
      const int64_t rounds = (wgs * sp + for_t + 255) / 256, it = (steps + sp * kw - 1) / (sp * kw);
      const bool full = M > 16 && M <= kMultiSmallM && rounds * 256 - wgs * sp < 16;
      const double us = rounds * (4.0 + it * per_step) + sp * M * N * 8 / 4.0e6 + (full ? 5.0 : 0.0);
      if (best.mt == 0 || us < least) {
        least = us;
        best = s;
        best.splits = (int)sp;
      }
    }
  }
  return best;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

int mid_tsplits(int64_t M, int64_t K) { return M <= kMultiSmallM ? (int)((K + kTSlice - 1) / kTSlice) : 0; }

size_t mid_fwd_bytes(int64_t M, int64_t N, int64_t K) {
  return up256((size_t)mid_shape(M, N, K).splits * M * N * 4) + (M <= kMultiSmallM ? up256((size_t)M * 4) : 0);
}

hipError_t launch_multi_final(const float *part, int splits, int64_t M, int64_t C, const MultiArgs &mu, uint16_t *out,
                              hipStream_t st) {
  const int64_t tiles = (M + 15) / 16;
  if (tiles > 65535 || (C & 7) != 0 || splits < 1) return hipErrorInvalidValue;
  MidArgs a{};
  a.M = M;
  a.N = C;
  a.Y = out;
  a.part = const_cast<float *>(part);
  a.splits = splits;
  launch_final(a, mu, st);
  return hipGetLastError();
}

hipError_t launch_mid_fwd_multi(const GemmArgs &ga, const MultiArgs &mu, const uint16_t *A, int ra, float *tpart,
                                int tsplits, uint16_t *T, float *part, hipStream_t st) {
  if ((ga.C & 7) != 0 || ga.ldo != ga.C || ga.M < 1 || ga.R % 64 != 0 || (mu.r & 7) != 0 || ra > mu.r || tsplits < 1)
    return hipErrorInvalidValue;
  const bool small = ga.M <= kMultiSmallM;
  const MidShape s = mid_shape(ga.M, ga.C, ga.R);
  const int64_t rows = (ga.M + 16 * s.mt - 1) / (16 * s.mt);
  const int64_t tiles = rows * ((ga.C + 32 * s.nw - 1) / (32 * s.nw)) * s.splits;
  const int64_t wgs = tiles + (small ? ga.M * ((mu.r + 31) / 32) * tsplits + (ga.M > 16) : 0);
  const int64_t frows = (ga.M + 15) / 16;
  int32_t *order = reinterpret_cast<int32_t *>(reinterpret_cast<char *>(part) + up256((size_t)s.splits * ga.M * ga.C * 4));
  if (wgs >= (int64_t(1) << 31) || frows > 65535 || (small && tsplits != mid_tsplits(ga.M, ga.R)))
    return hipErrorInvalidValue;
  const MidArgs a{ga.a_side, ga.w, ga.M, ga.C, ga.R, ga.out, part, s.splits, ga.t, tpart, tsplits, ra, T, (int)tiles,
                  A, order};
  const unsigned grid = (unsigned)wgs;
  switch (s.mt) {
#define MID_CASE(MT, NW, BLK)                            \
  case MT:                                               \
    if (s.al)                                            \
      launch_fmt<MT, NW, BLK, true>(a, mu, grid, st);    \
    else                                                 \
      launch_fmt<MT, NW, BLK, false>(a, mu, grid, st);   \
    break;
    MID_CASE(1, 4, 4) MID_CASE(2, 4, 4) MID_CASE(3, 8, 4) MID_CASE(4, 8, 4)
    MID_CASE(5, 8, 2) MID_CASE(6, 8, 2) MID_CASE(7, 8, 2) MID_CASE(8, 8, 2)
#undef MID_CASE
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  MultiArgs mf = mu;
  if (small) mf.perm = ga.M > 16 ? order : nullptr;
  launch_final(a, mf, st);
  return hipGetLastError();
}

}  // namespace nf4q
