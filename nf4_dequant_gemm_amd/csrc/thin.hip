// Both thin products of the backward pass over dY in one pass over it (gfx950, bf16 MFMA):
//
//   U = dY B  [M][r]     and     dB = s dY^T T  [N][r],   r <= 64
//
// for the layers that keep X in 8 bits. Each reads all of dY and little else, so the two launches of lora.hip cost
// two reads of it. Here a workgroup takes 256 or 512 rows and a range of columns, in steps of 128 columns that are staged in
// LDS once and multiplied twice: rows by B (U's sums over the range stay in registers until its end), and columns by T
// (dB's sums over the rows, written after each step). Sums over ranges and over row blocks are added in a
// fixed order by one further launch. T, a step of dY and of B are 122 KiB of LDS at rank 64, 158 of the CU's 160 with 512
// rows; at 128 they are more than there is, and the partials of dB, written and read, twice dY's bytes: above 64 the two
// launches stay.
//
// Bound by memory: a step's 64 KB are requested two steps ahead, 128 KB in flight on every CU. All of the adapters'
// gradients, k 512, against the two launches (us): 8192 x 14336 at rank 64 102 (117); 16384 x 14336 at 64 175 (232);
// 4096 x 11008 at 64 53 (68); 8192 x 14336 at 20 70 (98); 64 x 4096 at 16 24 (30). This kernel alone takes 97 us for 16384 x 11008 of 8
// experts at rank 16 (3.7 TB/s) and 57 for 8192 x 11008 at rank 64 (4.5 TB/s with its partials; 67 with blocks of 256
// rows). Two workgroups a CU with T in registers gained 5% at rank 16 where the order of steps gains 7.
#include "common.h"
#include "launch.h"
#include "sums.h"

#include <type_traits>

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
// kHalves: blocks of 256 rows that a workgroup takes one after the other at every step, whose sums of dB are one
// partial (2 without groups only: a group's blocks are numbered through all groups, and with every second workgroup idle 16384 x
// 11008 of 8 experts took 14 us more).
template <int TJ, bool kVec, bool kGrp, int kHalves>
__global__ __launch_bounds__(kT) void thin_kernel(const uint16_t *__restrict__ dy, const uint16_t *__restrict__ B,
                                                  const uint16_t *__restrict__ T, int64_t M, int64_t N, int r,
                                                  int64_t lsplit, int per, float *__restrict__ part_u,
                                                  float *__restrict__ part_b, GroupArgs gr) {
  constexpr int PROW = TJ * 16 + 8;             // row stride of T and B in bf16
  constexpr int CH = 2 * TJ;                    // 16-byte chunks of such a row
  __shared__ __align__(16) uint16_t sY[kRB * kYRow];
  __shared__ __align__(16) uint16_t sT[kHalves * kRB * PROW];
  __shared__ __align__(16) uint16_t sB[kCB * PROW];
  static_assert(sizeof(sY) + sizeof(sT) + sizeof(sB) <= 160 * 1024, "the LDS of a CU");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t blk = blockIdx.x;
  int64_t mbase = blk * kHalves * kRB, mhi = M;
  if (kGrp) {
    const int local = (int)blk * per;
    if (local >= grp_tile_off(gr, gr.E)) return;      // a grid sized by an upper bound
    const int e = find_group(gr, local);
    mbase = grp_m_off(gr, e) + (int64_t)((local - grp_tile_off(gr, e)) / per) * kRB;
    mhi = grp_m_off(gr, e + 1);
    B += e * N * r;
  }
  // the rows of a half
  auto rows = [&](int half) {
    const int64_t left = mhi - mbase - half * kRB;
    return left < 0 ? 0 : left < kRB ? left : kRB;
  };
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
  auto load = [&](auto half, int64_t l0, Stage &st) {
    const bool any = l0 < le;
    const __amdgpu_buffer_rsrc_t ry =
        make_rsrc(dy + (mbase + half * kRB) * N + l0, any && rows(half) ? (rows(half) * N - l0) * 2 : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = (tid + kT * i) >> 4, c = (tid & 15) * 8;
      st.y[i] = load16(ry, l0 + c < le ? (uint32_t)((row * N + c) * 2) : kNowhere);
    }
    if (half == 0) get(make_rsrc(B + l0 * r, any ? (le - l0) * r * 2 : 0), 0, st.b);
  };
  auto store = [&](auto half, const Stage &st) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<u32x4 *>(&sY[((tid + kT * i) >> 4) * kYRow + (tid & 15) * 8]) = st.y[i];
    if (half == 0) put(sB, st.b);
  };

  const int g16 = lane >> 4, l16 = lane & 15;
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(part_b + blk * r * N, (int64_t)r * N * 4);
  f32x4 u[kHalves * 2][TJ], d[TJ];
#pragma unroll
  for (int q = 0; q < kHalves * 2; ++q)
#pragma unroll
    for (int t = 0; t < TJ; ++t) u[q][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](auto half, int64_t l0) {
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
        for (int t = 0; t < TJ; ++t) u[half * 2 + q][t] = mfma16x16x32(y, b[t], u[half * 2 + q][t]);
      }
    }
    // dB: this wave's 16 columns by the 256 rows
    if (half == 0) {
#pragma unroll
      for (int t = 0; t < TJ; ++t) d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int k = 0; k < kRB / 32; ++k) {
      const bf16x8 y = columns(sY, kYRow, wave * 16, k, lane);
#pragma unroll
      for (int t = 0; t < TJ; ++t) d[t] = mfma16x16x32(columns(sT + half * kRB * PROW, PROW, t * 16, k, lane), y, d[t]);
    }
    if (half != kHalves - 1) return;
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
  constexpr std::integral_constant<int, 0> h0{};
  constexpr std::integral_constant<int, kHalves - 1> h1{};
  // The columns of an item: a step, or half of one. Row blocks begin at different steps, so that not all read the same
  // columns at a time: 16384 x 11008 at rank 16 166 us for 177, of 8 experts 97 for 104 (this kernel); blocks of 256 rows above
  // rank 32 lose by it (8192 x 11008 71 for 67).
  const int steps = (int)nst, turn = TJ == 4 && kHalves == 1 ? 0 : (int)blk % steps;
  auto at = [&](int i) {
    const int q = i / kHalves, c = q + turn;
    return q < steps ? lb + (int64_t)(c < steps ? c : c - steps) * kCB : le;
  };
  Stage s0, s1;
  {
    Narrow t[2 * kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const __amdgpu_buffer_rsrc_t rt = make_rsrc(T + (mbase + h * kRB) * r, rows(h) * r * 2);
      get(rt, 0, t[2 * h]);
      get(rt, 128, t[2 * h + 1]);
    }
    load(h0, at(0), s0);
    load(h1, at(1), s1);
#pragma unroll
    for (int h = 0; h < 2 * kHalves; ++h) put(sT + h * 128 * PROW, t[h]);
  }
  // items in pairs; one past the last is zeros and writes nothing
#pragma unroll 1
  for (int i = 0; i < steps * kHalves; i += 2) {
    store(h0, s0);
    __syncthreads();
    load(h0, at(i + 2), s0);
    step(h0, at(i));
    __syncthreads();
    store(h1, s1);
    __syncthreads();
    load(h1, at(i + 3), s1);
    step(h1, at(i + 1));
    __syncthreads();
  }
#pragma unroll
  for (int q = 0; q < kHalves * 2; ++q)
#pragma unroll
    for (int t = 0; t < TJ; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t row = mbase + q / 2 * kRB + wave * 32 + q % 2 * 16 + 4 * g16 + v;
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

template <int TJ, bool kVec, bool kGrp, int kHalves>
void launch_thin_as(const ThinArgs &a, const ThinPlan &p, float *part_b, const GroupArgs &gr, hipStream_t st) {
  thin_kernel<TJ, kVec, kGrp, kHalves><<<dim3((unsigned)p.blocks, (unsigned)p.splits), dim3(kT), 0, st>>>(
      a.dy, a.B, a.T, a.M, a.N, a.r, p.lsplit, a.per, a.part, part_b, gr);
}
template <int TJ>
void launch_thin(const ThinArgs &a, const ThinPlan &p, float *part_b, const GroupArgs &gr, hipStream_t st) {
  const bool vec = a.r % 8 == 0;
  if (gr.E) vec ? launch_thin_as<TJ, true, true, 1>(a, p, part_b, gr, st) : launch_thin_as<TJ, false, true, 1>(a, p, part_b, gr, st);
  else if (p.halves == 2) launch_thin_as<TJ, true, false, 2>(a, p, part_b, gr, st);
  else vec ? launch_thin_as<TJ, true, false, 1>(a, p, part_b, gr, st) : launch_thin_as<TJ, false, false, 1>(a, p, part_b, gr, st);
}

}  // namespace

ThinPlan thin_plan(int64_t M, int64_t N, int r, bool grouped, int E) {
  ThinPlan p;
  // Two blocks a workgroup halve the partials of dB where there are workgroups enough all the same (M N from 2^24 on),
  // the adapters' gradients with k 512 in us: 8192 x 14336 at rank 64 150 for 159, 16384 x 14336 222 for 250, 2048 x 11008 at 32
  // 42.7 for 46.4, 4096 x 11008 at 16 60.4 for 62.6; below, 1024 x 11008 at 32 would take 35.0 for 33.5, 2048 x 4096 at 64 42.8
  // for 37.9. Ranks that are not a multiple of 8 have no registers for it.
  p.halves = !grouped && r % 8 == 0 && M >= 4 * kRB && M * N >= (int64_t(1) << 24) ? 2 : 1;
  p.blocks = p.halves == 2 ? (M + 2 * kRB - 1) / (2 * kRB) : thin_blocks(M, E);
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
  const ThinPlan p = thin_plan(a.M, a.N, a.r, gr != nullptr, gr ? gr->E : 1);
  if (!thin_takes(a.M, a.N, a.r, gr ? gr->E : 1) || a.N % 8 || a.N > (int64_t(1) << 22) || p.blocks < 1 || p.splits > 65535) return hipErrorInvalidValue;
  float *part_b = a.part + p.u_floats;
  const GroupArgs groups = gr ? *gr : GroupArgs{};
  if (a.r <= 16) launch_thin<1>(a, p, part_b, groups, st);
  else if (a.r <= 32) launch_thin<2>(a, p, part_b, groups, st);
  else launch_thin<4>(a, p, part_b, groups, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int threads = split_sum_t_threads(a.r);
  const int64_t cb = (a.N + 63) / 64, ub = (a.M * a.r + threads - 1) / threads;
  thin_final_kernel<<<dim3((unsigned)(cb * (gr ? gr->E : 1) + (ub < 1024 ? ub : 1024))), dim3(threads), 0, st>>>(
      a, part_b, (int)p.blocks, p.splits, (int)cb, groups);
  return hipGetLastError();
}

}  // namespace nf4q
