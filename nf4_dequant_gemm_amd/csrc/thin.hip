// Both thin products of the backward pass over dY in one pass over it (gfx950, bf16 MFMA):
//
//   U = dY B  [M][r]     and     dB = s dY^T T  [N][r],   r <= 64
//
// for the layers that keep X in 8 bits. Each reads all of dY and little else, so the two launches of lora.hip cost
// two reads of it. Here a workgroup takes 256 rows and a range of columns, in steps of 128 columns that are staged in
// LDS once and multiplied twice: rows by B (U's sums over the range stay in registers until its end), and columns by T
// (dB's sums over the 256 rows, written after each step). Sums over ranges and over row blocks are added in a
// fixed order by one further launch. T, a step of dY and of B are 125 KB of LDS at rank 64; at 128 they are more than
// there is, and the partials of dB, written and read, twice dY's bytes: above 64 the two launches stay.
//
// Bound by memory: a step's 64 KB are requested two steps ahead, 128 KB in flight on every CU. All of the adapters'
// gradients, k 512, against the two launches: 8192 x 14336 at rank 64 163 us (180), 48 155 (171), 40 148 (168);
// 16384 x 14336 at 64 255 (290); 4096 x 11008 at 64 86 (98), at 8 63 (78); 64 x 4096 at 16 21 (27). This kernel alone
// takes 105 us for 16384 x 11008 of 8 experts at rank 16 (3.4 TB/s; 116 with ranges of columns sized for the fullest
// rounds alone), and 67 for 8192 x 11008 at rank 64 with half as many bytes of partials (4.0 TB/s). Two workgroups a
// CU with T in registers at rank 16 took 100, steps in another order for each row block 98 there and 71 for 67 here.
#include "common.h"
#include "launch.h"
#include "sums.h"

namespace nf4q {
namespace {

constexpr int kRB = kThinRows, kCB = 128, kT = 512;
constexpr int kYRow = kCB + 8;                  // dY row stride in bf16: 16 rows' chunks in different banks
constexpr uint32_t kNowhere = 0x80000000u;      // an offset past every buffer: reads 0
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0);
}
__device__ __forceinline__ uint16_t load2(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, offset, 0, 0);
}
__device__ __forceinline__ s16x4 lds_tr16(const uint16_t *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}
// 8 consecutive rows (of slice k of 32) of column col + lane % 16 of a row-major LDS tile: a matrix operand whose
// reduction runs over the rows.
__device__ __forceinline__ bf16x8 columns(const uint16_t *tile, int stride, int col, int k, int lane) {
  const uint16_t *p = tile + (k * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2)) * stride + col + 4 * (lane & 3);
  const s16x4 a = lds_tr16(p), b = lds_tr16(p + 4 * stride);
  return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// kVec: r is a multiple of 8. kGrp: rows grouped by expert; B is the expert's, and row blocks are counted through
// gr.tile_off, which holds them times `per`.
template <int TJ, bool kVec, bool kGrp>
__global__ __launch_bounds__(kT) void thin_kernel(const uint16_t *__restrict__ dy, const uint16_t *__restrict__ B,
                                                  const uint16_t *__restrict__ T, int64_t M, int64_t N, int r,
                                                  int64_t lsplit, int per, float *__restrict__ part_u,
                                                  float *__restrict__ part_b, GroupArgs gr) {
  constexpr int PROW = TJ * 16 + 8;             // row stride of T and B in bf16
  constexpr int CH = 2 * TJ;                    // 16-byte chunks of such a row
  __shared__ __align__(16) uint16_t sY[kRB * kYRow];
  __shared__ __align__(16) uint16_t sT[kRB * PROW];
  __shared__ __align__(16) uint16_t sB[kCB * PROW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t blk = blockIdx.x;
  int64_t mbase = blk * kRB, mhi = M;
  if (kGrp) {
    const int local = (int)blk * per;
    if (local >= grp_tile_off(gr, gr.E)) return;      // a grid sized by an upper bound
    const int e = find_group(gr, local);
    mbase = grp_m_off(gr, e) + (int64_t)((local - grp_tile_off(gr, e)) / per) * kRB;
    mhi = grp_m_off(gr, e + 1);
    B += e * N * r;
  }
  const int64_t rows = mhi - mbase < kRB ? mhi - mbase : kRB;
  const int split = blockIdx.y;
  const int64_t lb = split * lsplit, le = lb + lsplit < N ? lb + lsplit : N;

  // rows of a matrix [.][r] in LDS rows of PROW: 16-byte chunks, or element by element
  constexpr int NV = TJ > 2 ? 2 : 1;
  struct Narrow {
    u32x4 v[NV];
    uint16_t e[kVec ? 1 : 4 * TJ];
  };
  auto get = [&](__amdgpu_buffer_rsrc_t rs, int first, Narrow &x) {     // 128 rows from `first` on
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int row = (tid + kT * i) / CH, j = (tid + kT * i) % CH * 8;
        x.v[i] = load16(rs, row < 128 && j < r ? (uint32_t)(((first + row) * r + j) * 2) : kNowhere);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * TJ; ++i) {
        const int row = (tid + kT * i) / (16 * TJ), j = (tid + kT * i) % (16 * TJ);
        x.e[i] = load2(rs, j < r ? (uint32_t)(((first + row) * r + j) * 2) : kNowhere);
      }
    }
  };
  auto put = [&](uint16_t *tile, const Narrow &x) {
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int row = (tid + kT * i) / CH;
        if (row < 128) *reinterpret_cast<u32x4 *>(&tile[row * PROW + (tid + kT * i) % CH * 8]) = x.v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * TJ; ++i) tile[(tid + kT * i) / (16 * TJ) * PROW + (tid + kT * i) % (16 * TJ)] = x.e[i];
    }
  };

  struct Stage {
    u32x4 y[8];
    Narrow b;
  };
  // Requests a step, without a branch (a skipped request would make the waits for the step before wait for this
  // one's too): rows and columns outside read as zeros.
  auto load = [&](int64_t l0, Stage &st) {
    const bool any = l0 < le;
    const __amdgpu_buffer_rsrc_t ry = make_rsrc(dy + mbase * N + l0, any ? (rows * N - l0) * 2 : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = (tid + kT * i) >> 4, c = (tid & 15) * 8;
      st.y[i] = load16(ry, l0 + c < le ? (uint32_t)((row * N + c) * 2) : kNowhere);
    }
    get(make_rsrc(B + l0 * r, any ? (le - l0) * r * 2 : 0), 0, st.b);
  };
  auto store = [&](const Stage &st) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<u32x4 *>(&sY[((tid + kT * i) >> 4) * kYRow + (tid & 15) * 8]) = st.y[i];
    put(sB, st.b);
  };

  const int g16 = lane >> 4, l16 = lane & 15;
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(part_b + blk * r * N, (int64_t)r * N * 4);
  f32x4 u[2][TJ];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int t = 0; t < TJ; ++t) u[q][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](int64_t l0) {
    // U: this wave's 32 rows by the step's 128 columns
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      bf16x8 b[TJ];
#pragma unroll
      for (int t = 0; t < TJ; ++t) b[t] = columns(sB, PROW, t * 16, k, lane);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bf16x8 y = __builtin_bit_cast(
            bf16x8, *reinterpret_cast<const u32x4 *>(&sY[(wave * 32 + q * 16 + l16) * kYRow + k * 32 + g16 * 8]));
#pragma unroll
        for (int t = 0; t < TJ; ++t) u[q][t] = mfma16x16x32(y, b[t], u[q][t]);
      }
    }
    // dB: this wave's 16 columns by the 256 rows
    f32x4 d[TJ];
#pragma unroll
    for (int t = 0; t < TJ; ++t) d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kRB / 32; ++k) {
      const bf16x8 y = columns(sY, kYRow, wave * 16, k, lane);
#pragma unroll
      for (int t = 0; t < TJ; ++t) d[t] = mfma16x16x32(columns(sT, PROW, t * 16, k, lane), y, d[t]);
    }
    const int64_t c = l0 + wave * 16 + l16;
#pragma unroll
    for (int t = 0; t < TJ; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int j = t * 16 + 4 * g16 + v;
        // dropped outside; without a branch for the same reason as the requests
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(d[t][v]), rb,
                                              j < r && c < le ? (uint32_t)((j * N + c) * 4) : kNowhere, 0, 0);
      }
  };

  const int64_t nst = le > lb ? (le - lb + kCB - 1) / kCB : 0;
  if (nst == 0) return;       // the whole workgroup
  Stage s0, s1;
  {
    Narrow t0, t1;
    const __amdgpu_buffer_rsrc_t rt = make_rsrc(T + mbase * r, rows * r * 2);
    get(rt, 0, t0);
    get(rt, 128, t1);
    load(lb, s0);
    load(lb + kCB, s1);
    put(sT, t0);
    put(sT + 128 * PROW, t1);
  }
  // steps in pairs; one past the last is zeros and writes nothing
#pragma unroll 1
  for (int64_t i = 0; i < nst; i += 2) {
    store(s0);
    __syncthreads();
    load(lb + (i + 2) * kCB, s0);
    step(lb + i * kCB);
    __syncthreads();
    store(s1);
    __syncthreads();
    load(lb + (i + 3) * kCB, s1);
    step(lb + (i + 1) * kCB);
    __syncthreads();
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int t = 0; t < TJ; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t row = mbase + wave * 32 + q * 16 + 4 * g16 + v;
        const int j = t * 16 + l16;
        if (row < mhi && j < r) part_u[((int64_t)split * M + row) * r + j] = u[q][t][v];
      }
}

// The sums of the partials, one launch for both: workgroups below cb * E take 64 of the cb * 64 columns of an expert's dB
// (E = 1 without groups) from its row blocks, the others U.
__global__ __launch_bounds__(1024) void thin_final_kernel(ThinArgs a, const float *__restrict__ part_b, int blocks,
                                                          int splits, int cb, GroupArgs gr) {
  const int E = gr.E ? gr.E : 1;
  if ((int)blockIdx.x >= cb * E) {
    split_sum_each(a.part, a.M * a.r, splits, a.U, a.Uw, (int)blockIdx.x - cb * E, (int)gridDim.x - cb * E);
    return;
  }
  const int e = (int)blockIdx.x / cb;
  int first = 0, count = blocks;
  if (gr.E) {
    first = grp_tile_off(gr, e) / a.per;
    count = grp_tile_off(gr, e + 1) / a.per - first;
  }
  split_sum_t(part_b + (int64_t)first * a.r * a.N, a.N, a.r, count, a.s, a.dB + (int64_t)e * a.r * a.N,
              (int64_t)((int)blockIdx.x % cb) * 64);
}

template <int TJ, bool kVec>
void launch_thin_as(const ThinArgs &a, const ThinPlan &p, float *part_b, const GroupArgs *gr, hipStream_t st) {
  const dim3 grid((unsigned)p.blocks, (unsigned)p.splits);
  if (gr) thin_kernel<TJ, kVec, true><<<grid, dim3(kT), 0, st>>>(a.dy, a.B, a.T, a.M, a.N, a.r, p.lsplit, a.per, a.part,
                                                                 part_b, *gr);
  else thin_kernel<TJ, kVec, false><<<grid, dim3(kT), 0, st>>>(a.dy, a.B, a.T, a.M, a.N, a.r, p.lsplit, 1, a.part, part_b,
                                                               GroupArgs{});
}

}  // namespace

ThinPlan thin_plan(int64_t M, int64_t N, int r, int E) {
  ThinPlan p;
  p.blocks = thin_blocks(M, E);
  // ranges of columns of equally many steps (the last one fewer), at least two as the loop takes pairs: the rounds of
  // 256 workgroups times the steps of one, and one more for its first requests, least
  const int64_t steps = (N + kCB - 1) / kCB;
  int64_t best = steps, cost = INT64_MAX;
  for (int64_t len = steps < 128 ? steps : 128; len >= 2; --len) {
    const int64_t rounds = (p.blocks * ((steps + len - 1) / len) + 255) / 256;
    if (rounds * (len + 1) < cost) cost = rounds * (len + 1), best = len;
  }
  p.lsplit = best * kCB;
  p.splits = (int)((N + p.lsplit - 1) / p.lsplit);
  p.u_floats = ((size_t)p.splits * M * r + 63) / 64 * 64;      // the other partials behind them aligned
  p.b_floats = (size_t)p.blocks * r * N;
  return p;
}

hipError_t launch_thin_bwd(const ThinArgs &a, const GroupArgs *gr, hipStream_t st) {
  const ThinPlan p = thin_plan(a.M, a.N, a.r, gr ? gr->E : 1);
  if (!thin_takes(a.M, a.N, a.r, gr ? gr->E : 1) || a.N % 8 || a.N > (int64_t(1) << 22) || p.blocks < 1 || p.splits > 65535) return hipErrorInvalidValue;
  float *part_b = a.part + p.u_floats;
  if (a.r <= 16) {
    if (a.r & 7) launch_thin_as<1, false>(a, p, part_b, gr, st);
    else launch_thin_as<1, true>(a, p, part_b, gr, st);
  } else if (a.r <= 32) {
    if (a.r & 7) launch_thin_as<2, false>(a, p, part_b, gr, st);
    else launch_thin_as<2, true>(a, p, part_b, gr, st);
  } else {
    if (a.r & 7) launch_thin_as<4, false>(a, p, part_b, gr, st);
    else launch_thin_as<4, true>(a, p, part_b, gr, st);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int threads = split_sum_t_threads(a.r);
  const int64_t cb = (a.N + 63) / 64, ub = (a.M * a.r + threads - 1) / threads;
  thin_final_kernel<<<dim3((unsigned)(cb * (gr ? gr->E : 1) + (ub < 1024 ? ub : 1024))), dim3(threads), 0, st>>>(
      a, part_b, (int)p.blocks, p.splits, (int)cb, gr ? *gr : GroupArgs{});
  return hipGetLastError();
}

}  // namespace nf4q
