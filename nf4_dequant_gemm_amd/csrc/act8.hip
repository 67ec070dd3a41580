// Activations kept in 8 bits for the backward pass (gfx950).
//
// A row is cut into blocks of 64 elements (the last may be short; code rows are padded with zeros to a
// multiple of 64). With a = max |x| of a block,
//
//   code = 127 x / a rounded to the nearest integer, ties to even;   scale = fl32(a / 127)
//
// and the block stands for fl32(code scale): at most a / 254 (half a step) from x, up to the rounding of
// the scale (at the largest float32 the scale is cut so that 127 of it stay finite). A block whose a is below
// 2^-119 is stored as zeros, so that 127 / a is finite; one with an Inf or NaN gets the scale NaN, so that
// whatever uses it is NaN.
//
// act8_pack and act8_unpack read and write each element once and are bound by memory. Where the layer's
// backward pass uses the kept activation, the codes are read in its place, decoded on the way into the
// matrix cores or the activation's derivative, and never expanded in memory.
//
// Measured: 16384 x 14336 in bf16 packed in 133 us and unpacked in 137 us (719 MB each, 5.3 TB/s).
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace nf4q {
namespace {

typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;

// ---------------------------------------------------------------------------------- pack, unpack
// The 16 elements of a thread as words (bf16 pairs, or float32).
template <typename XT>
struct Piece {
  static constexpr int kWords = 16 * (int)sizeof(XT) / 4;
  uint32_t w[kWords];
};

// Bits of the largest |x| (as of float32): an unsigned maximum, in which Inf and NaN come last.
__device__ __forceinline__ uint32_t top_bits(const Piece<uint16_t> &p) {
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, p.w[i] & 0x7FFF7FFFu));
  return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
}
__device__ __forceinline__ uint32_t top_bits(const Piece<float> &p) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t b = p.w[i] & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
  return m;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The code of a float32 x whose 127 x / a may lie too close to a border for float32: compared there with
// the border in float64, where both sides are exact.
__device__ __forceinline__ int code_at_border(float x, float a, float t) {
  const double h = floor(fabs((double)t));              // between h and h + 1, |t| near h + 1/2
  const double d = 254.0 * fabs((double)x) - (2.0 * h + 1.0) * (double)a;
  const int c = (int)h + (d > 0.0 || (d == 0.0 && ((int)h & 1)) ? 1 : 0);
  return x < 0.f ? -c : c;
}

// Codes by one fused multiply-add each: x inv + 1.5 2^23 is rounded, ties to even, at the integers, which
// leaves the code in the low bits. inv is 127 / a rounded up. For bf16 x and a that gives the exact code:
// 127 x / a differs from a half-integer, if at all, by more than 2^-17 of itself (its distance times 2 a is
// an integer multiple of the last bits of both 8-bit significands), far above the 2^-23 of inv; and where it
// is a half-integer, either 127 / a is exact (a = 127 2^i) and the tie goes to even, or x = +-a / 2, and the
// rounded-up inv takes 63.5 to 64, which is even.
constexpr float kRound = 12582912.f;
constexpr float kTopScale = 0x1.020406p+121f;     // the largest whose 127-fold is finite

template <typename XT>
__device__ __forceinline__ uint32_t four_codes(const Piece<XT> &p, int i, float inv, float a) {
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(XT) == 2) {
      const uint32_t w = p.w[2 * i + (e >> 1)];
      c[e] = __float_as_uint(__builtin_fmaf((e & 1) ? bf16_hi(w) : bf16_lo(w), inv, kRound));
    } else {
      const float x = __uint_as_float(p.w[4 * i + e]);
      c[e] = __float_as_uint(__builtin_fmaf(x, inv, kRound));
      // t is off by at most 2^-15; rare (about 2^-14 of the elements), so the branch costs next to nothing
      const float t = x * inv;
      if (fabsf(fabsf(t - rintf(t)) - 0.5f) < 0x1p-14f) c[e] = (uint32_t)code_at_border(x, a, t);
    }
  }
  return perm(perm(c[3], c[2], 0x0C0C0400u), perm(c[1], c[0], 0x0C0C0400u), 0x05040100u);
}

// 16 bytes in memory, aligned to that (kVec) or to their elements.
typedef u32x4 __attribute__((aligned(2))) u32x4_by2;
typedef u32x4 __attribute__((aligned(4))) u32x4_by4;
template <typename XT, bool kVec>
using Mem16 = std::conditional_t<kVec, u32x4, std::conditional_t<sizeof(XT) == 2, u32x4_by2, u32x4_by4>>;

// A thread packs 16 elements; four lanes make a block. kVec: k, ldx and the base are multiples of 16 bytes;
// otherwise rows lie at any alignment and the last chunk of a row may be short.
template <typename XT, bool kVec>
__global__ __launch_bounds__(256) void act8_pack_kernel(const XT *__restrict__ x, int64_t ldx, Act8 q) {
  const uint32_t pieces = (uint32_t)(q.kp / 16);
  const int64_t first = (int64_t)blockIdx.x * 256, row0 = first / pieces;
  const uint32_t at = (uint32_t)(first - row0 * pieces) + threadIdx.x;
  const int64_t row = row0 + at / pieces;
  const int64_t c = (int64_t)(at % pieces) * 16;
  const bool live = row < q.rows;         // whole blocks of four lanes
  Piece<XT> p;
  const XT *src = x + row * ldx + c;
  constexpr int P = 16 / (int)sizeof(XT);
#pragma unroll
  for (int i = 0; i < 16 / P; ++i) {
    u32x4 v = {0, 0, 0, 0};
    const int64_t left = live ? q.k - c - i * P : 0;
    if (kVec ? left > 0 : left >= P) {
      v = *reinterpret_cast<const Mem16<XT, kVec> *>(src + i * P);
    } else if constexpr (!kVec) {
#pragma unroll
      for (int e = 0; e < P - 1; ++e)
        if (e < left) {
          if constexpr (sizeof(XT) == 2) v[e >> 1] |= (uint32_t)src[i * P + e] << (16 * (e & 1));
          else v[e] = __float_as_uint(src[i * P + e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) p.w[4 * i + e] = v[e];
  }
  uint32_t m = top_bits(p);
  m = umax(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));   // lanes 1, 0, 3, 2
  m = umax(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));   // lanes 2, 3, 0, 1
  if (!live) return;
  const float a = __uint_as_float(m);
  u32x4 codes = {0, 0, 0, 0};
  float scale = 0.f;
  if (m >= 0x7F800000u) {
    scale = __uint_as_float(0x7FC00000u);
  } else if (a >= 0x1p-119f) {
    scale = fminf(a / 127.f, kTopScale);
    float inv = 127.f / a;
    if (__builtin_fmaf(-inv, a, 127.f) > 0.f) inv = __uint_as_float(__float_as_uint(inv) + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) codes[i] = four_codes<XT>(p, i, inv, a);
  }
  *reinterpret_cast<u32x4 *>(q.codes + row * q.kp + c) = codes;
  if ((threadIdx.x & 3) == 0) q.scale[row * (q.kp / kAct8Block) + c / kAct8Block] = scale;
}

// What code e of a word of codes stands for.
__device__ __forceinline__ float code_value(uint32_t codes, int e, float scale) {
  return (float)(int8_t)(codes >> (8 * e)) * scale;
}

template <typename XT, bool kVec>
__global__ __launch_bounds__(256) void act8_unpack_kernel(Act8 q, XT *__restrict__ x, int64_t ldx) {
  const uint32_t pieces = (uint32_t)(q.kp / 16);
  const int64_t first = (int64_t)blockIdx.x * 256, row0 = first / pieces;
  const uint32_t at = (uint32_t)(first - row0 * pieces) + threadIdx.x;
  const int64_t row = row0 + at / pieces;
  const int64_t c = (int64_t)(at % pieces) * 16;
  if (row >= q.rows) return;
  const u32x4 codes = *reinterpret_cast<const u32x4 *>(q.codes + row * q.kp + c);
  const float scale = q.scale[row * (q.kp / kAct8Block) + c / kAct8Block];
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = code_value(codes[e >> 2], e & 3, scale);
  XT *dst = x + row * ldx + c;
  constexpr int P = 16 / (int)sizeof(XT);
#pragma unroll
  for (int i = 0; i < 16 / P; ++i) {
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(XT) == 2) o[e] = pack_bf16x2(v[P * i + 2 * e], v[P * i + 2 * e + 1]);
      else o[e] = __float_as_uint(v[P * i + e]);
    }
    const int64_t left = q.k - c - i * P;
    if (kVec ? left > 0 : left >= P) {
      *reinterpret_cast<Mem16<XT, kVec> *>(dst + i * P) = o;
    } else if constexpr (!kVec) {
#pragma unroll
      for (int e = 0; e < P - 1; ++e)
        if (e < left) {
          if constexpr (sizeof(XT) == 2) dst[i * P + e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
          else dst[i * P + e] = __uint_as_float(o[e]);
        }
    }
  }
}

// ---------------------------------------------------------------------------------- sums over rows
// out[j][c] = sum over m of P[m][j] Q[m][c], P float32, Q = code x scale in 8 bits. The scale of a row's block of 64
// columns goes to P: for each of its blocks a workgroup holds bf16(P scale) of the stage's rows, and the codes,
// which bf16 holds exactly, are multiplied as they are. So the one rounding before the float32 sums is that of
// P scale, and a code costs one and a half vector instructions (a conversion with byte select and sign
// extension, half a conversion of a pair). With the scale applied to the codes it was two and a half, and with
// P's rounding made up for by a second bf16 number twice the products (16384 x 14336, rank 32: 72 us). Now that
// case takes 67 us and 8192 x 4096, rank 64, 16.5 us, most of it memory: without the products 61 us.
//
// Workgroup: 32 NW columns x all r (<= 128) rows j over one split of the rows, in stages of 64 rows requested two
// stages ahead. The codes stay bytes in LDS and are read with the transposing load ds_read_b64_tr_b8, which
// hands each lane 8 consecutive rows of one column, the matrix cores' operand layout.
constexpr int kBM = 64;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((ext_vector_type(2))) int i32x2;

__device__ __forceinline__ s16x4 lds_tr16(const uint16_t *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}
__device__ __forceinline__ u32x2 lds_tr8(const int8_t *p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2 *)(p)));
}

// Waves of a workgroup for TJ tiles of 16 ranks: with 8, the four blocks' P takes too much LDS above 64 ranks.
constexpr int act8_waves(int tj) { return tj <= 4 ? 8 : 4; }

// kPVec: r is a multiple of 4. kGrp: one sum for each expert blockIdx.z over its own rows. kMap: row m is row map[m]
// of q (zeros where that is not one of its rows).
template <int TJ, bool kPVec, bool kGrp, bool kMap>
__device__ __forceinline__ void mreduce_act8_body(const float *__restrict__ P, const Act8 &q, const int *__restrict__ map,
                                                  int64_t M, int r, int64_t msplit, float *__restrict__ part,
                                                  const GroupArgs &gr) {
  constexpr int NW = act8_waves(TJ), NB = NW / 2;     // waves; blocks of 64 columns
  constexpr int kT = 64 * NW, kBC = 32 * NW;          // threads, columns
  constexpr int PROW = TJ * 16 + 8;                   // P row stride in bf16
  constexpr int kQRow = kBC + 16;                     // code row stride: 8 rows in different banks
  constexpr int PC = 4 * TJ;                          // 16-byte chunks of a row of P
  constexpr int PPT = (kBM * PC + kT - 1) / kT;       // chunks of P a thread (past row 63: read as any, not stored)
  constexpr uint32_t kNowhere = 0x80000000u;          // an offset past every buffer: reads 0
  __shared__ __align__(16) int8_t sQ[2][kBM * kQRow];
  __shared__ __align__(16) uint16_t sP[2][NB][kBM * PROW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // Workgroups go to the 8 XCDs in turn: each takes neighbouring column tiles of the same rows, which share
  // lines of scales and P in its L2.
  const int total = gridDim.x * gridDim.y, id = blockIdx.y * gridDim.x + blockIdx.x, per = total / 8, more = total % 8;
  const int x = id % 8, at = x * per + (x < more ? x : more) + id / 8;
  const int64_t c0 = (int64_t)(at % gridDim.x) * kBC, C = q.k;
  const int split = at / gridDim.x;
  int64_t lo = 0, hi = M;
  if (kGrp) {
    lo = grp_m_off(gr, blockIdx.z);
    hi = grp_m_off(gr, blockIdx.z + 1);
    msplit = (hi - lo + gridDim.y - 1) / gridDim.y;
    msplit = (msplit + kBM - 1) / kBM * kBM;
  }
  const int64_t mb = lo + split * msplit;
  const int64_t me = (mb + msplit < hi) ? mb + msplit : hi;
  const int64_t kp = q.kp, nb = kp / kAct8Block, b0 = c0 / kAct8Block;

  f32x4 acc[TJ][2];
#pragma unroll
  for (int t = 0; t < TJ; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};

  // A thread's part of a stage: 16 codes of rows tid / (2 NW) and 32 rows on, columns c0 + 16 (tid % (2 NW)); chunks
  // of four ranks of P, row (tid + kT i) / PC, with the scales of that row's blocks.
  const int qr = tid / (2 * NW), qc = tid % (2 * NW) * 16;
  const bool q_in = c0 + qc < kp;
  const uint32_t q_off = q_in ? (uint32_t)(qr * kp + c0 + qc) : kNowhere;
  const uint32_t q_off2 = q_in ? (uint32_t)((qr + 32) * kp + c0 + qc) : kNowhere;
  auto p_row = [&](int i) { return (tid + kT * i) / PC; };
  auto p_col = [&](int i) { return (tid + kT * i) % PC * 4; };

  struct Stage {
    u32x4 q[2];
    f32x4 p[PPT];
    float s[PPT][NB];
  };
  struct Rows {       // kMap: the rows of q of this thread's codes and chunks of P, -1 past the split's end
    int q[2], p[PPT];
  };
  auto find = [&](int64_t ms, Rows &rw) {
    const int left = me > ms ? me - ms < kBM ? (int)(me - ms) : kBM : 0;
    const __amdgpu_buffer_rsrc_t rm = make_rsrc(map + ms, left * 4);
    // past the end the buffer reads as 0, which is a row of q: its scale may be NaN, and P's zeros would not hide it
    auto of = [&](int row) {
      const int at = (int)__builtin_amdgcn_raw_buffer_load_b32(rm, row * 4, 0, 0);
      return row < left ? at : -1;
    };
    rw.q[0] = of(qr);
    rw.q[1] = of(qr + 32);
#pragma unroll
    for (int i = 0; i < PPT; ++i) rw.p[i] = of(p_row(i));
  };
  // Requests a stage, without a branch: the waits for the stage before then leave these requests in flight. Rows
  // past the split's end read as zeros (of P too); a row of q that is none as row 0 with the scale 0.
  auto load = [&](int64_t ms, Stage &st, const Rows &rw) {
    const int64_t left = me > ms ? me - ms < kBM ? me - ms : kBM : 0;
    if constexpr (kMap) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = rw.q[i] >= 0 && rw.q[i] < q.rows ? rw.q[i] : 0;
        st.q[i] = *reinterpret_cast<const u32x4 *>(q.codes + row * kp + (q_in ? c0 + qc : 0));
      }
    } else {
      const __amdgpu_buffer_rsrc_t rq = make_rsrc(q.codes + ms * kp, left * kp);
      st.q[0] = __builtin_amdgcn_raw_buffer_load_b128(rq, q_off, 0, 0);
      st.q[1] = __builtin_amdgcn_raw_buffer_load_b128(rq, q_off2, 0, 0);
    }
    const __amdgpu_buffer_rsrc_t rp = make_rsrc(P + ms * r, left * r * 4);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(q.scale + (kMap ? 0 : ms * nb), kMap ? 0 : left * nb * 4);
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      const int row = p_row(i), j = p_col(i);
      if constexpr (kPVec) {
        st.p[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                rp, j < r ? (uint32_t)((row * r + j) * 4) : kNowhere, 0, 0));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st.p[i][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
              rp, j + e < r ? (uint32_t)((row * r + j + e) * 4) : kNowhere, 0, 0));
      }
      // the scales of the row's blocks; past the row's last block any value will do (no column uses it)
      if constexpr (kMap) {
        const bool in = rw.p[i] >= 0 && rw.p[i] < q.rows;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float v = q.scale[(in ? rw.p[i] : 0) * nb + (b0 + b < nb ? b0 + b : 0)];
          st.s[i][b] = in ? v : 0.f;
        }
      } else if constexpr (NB == 4) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, (uint32_t)((row * nb + b0) * 4), 0, 0);
#pragma unroll
        for (int b = 0; b < 4; ++b) st.s[i][b] = __uint_as_float(v[b]);
      } else {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs, (uint32_t)((row * nb + b0) * 4), 0, 0);
#pragma unroll
        for (int b = 0; b < 2; ++b) st.s[i][b] = __uint_as_float(v[b]);
      }
    }
  };
  auto store = [&](const Stage &st, int buf) {
    *reinterpret_cast<u32x4 *>(&sQ[buf][qr * kQRow + qc]) = st.q[0];
    *reinterpret_cast<u32x4 *>(&sQ[buf][(qr + 32) * kQRow + qc]) = st.q[1];
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      if (kBM * PC % kT != 0 && p_row(i) >= kBM) continue;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float s = st.s[i][b];
        const u32x2 v = {pack_bf16x2(st.p[i][0] * s, st.p[i][1] * s), pack_bf16x2(st.p[i][2] * s, st.p[i][3] * s)};
        *reinterpret_cast<u32x2 *>(&sP[buf][b][p_row(i) * PROW + p_col(i)]) = v;
      }
    }
  };
  const int g16 = lane >> 4, l16 = lane & 15;
  auto mma = [&](int buf) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int m0 = ks * 32 + g16 * 8;        // this lane's 8 rows
      bf16x8 bq[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const u32x2 w = lds_tr8(&sQ[buf][(m0 + (l16 >> 1)) * kQRow + wave * 32 + u * 16 + (l16 & 1) * 8]);
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = pack_bf16x2((float)(int8_t)(w[e >> 1] >> (16 * (e & 1))), (float)(int8_t)(w[e >> 1] >> (16 * (e & 1) + 8)));
        bq[u] = __builtin_bit_cast(bf16x8, v);
      }
#pragma unroll
      for (int t = 0; t < TJ; ++t) {
        const uint16_t *S = &sP[buf][wave >> 1][(m0 + (l16 >> 2)) * PROW + t * 16 + 4 * (l16 & 3)];
        const s16x4 a = lds_tr16(S), b = lds_tr16(S + 4 * PROW);
        const bf16x8 ap = __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
#pragma unroll
        for (int u = 0; u < 2; ++u) acc[t][u] = mfma16x16x32(ap, bq[u], acc[t][u]);
      }
    }
  };

  // stage i: products on buffer i & 1; requests of stage i + 2 (and of the rows of stage i + 4); stores of stage
  // i + 1. A stage past the last is zeros, so the stages are taken in pairs.
  const int64_t nst = (me > mb) ? (me - mb + kBM - 1) / kBM : 0;
  if (nst > 0) {
    Stage s0, s1;
    Rows r0{}, r1{};
    if constexpr (kMap) {
      find(mb, r0);
      find(mb + kBM, r1);
    }
    load(mb, s0, r0);
    load(mb + kBM, s1, r1);
    if constexpr (kMap) {
      find(mb + 2 * kBM, r0);
      find(mb + 3 * kBM, r1);
    }
    store(s0, 0);
    __syncthreads();
#pragma unroll 1
    for (int64_t i = 0; i < nst; i += 2) {
      load(mb + (i + 2) * kBM, s0, r0);
      if constexpr (kMap) find(mb + (i + 4) * kBM, r0);
      mma(0);
      store(s1, 1);
      __syncthreads();
      load(mb + (i + 3) * kBM, s1, r1);
      if constexpr (kMap) find(mb + (i + 5) * kBM, r1);
      mma(1);
      store(s0, 0);
      __syncthreads();
    }
  }

#pragma unroll
  for (int t = 0; t < TJ; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int j = t * 16 + 4 * g16 + v;
        const int64_t c = c0 + wave * 32 + u * 16 + l16;
        if (j < r && c < C) part[(((int64_t)blockIdx.z * gridDim.y + split) * r + j) * C + c] = acc[t][u][v];
      }
}

template <int TJ, bool kPVec>
__global__ __launch_bounds__(64 * act8_waves(TJ)) void mreduce_act8_kernel(const float *__restrict__ P, Act8 q, int64_t M,
                                                                           int r, int64_t msplit,
                                                                           float *__restrict__ part) {
  mreduce_act8_body<TJ, kPVec, false, false>(P, q, nullptr, M, r, msplit, part, GroupArgs{});
}

template <int TJ, bool kPVec, bool kMap>
__global__ __launch_bounds__(64 * act8_waves(TJ)) void mreduce_act8_grouped_kernel(const float *__restrict__ P, Act8 q,
                                                                                   const int *__restrict__ map, int r,
                                                                                   float *__restrict__ part,
                                                                                   GroupArgs gr) {
  mreduce_act8_body<TJ, kPVec, true, kMap>(P, q, map, 0, r, 0, part, gr);
}

// The launch for one height and kind of P.
template <int TJ, bool kPVec>
hipError_t launch_mreduce_act8_as(const float *P, const Act8 &q, const int *map, int64_t M, int r, int splits,
                                  float *part, const GroupArgs *gr, hipStream_t st) {
  constexpr int kBC = 32 * act8_waves(TJ);
  const dim3 grid((unsigned)((q.k + kBC - 1) / kBC), (unsigned)splits, (unsigned)(gr ? gr->E : 1));
  const dim3 block(64 * act8_waves(TJ));
  int64_t msplit = (M + splits - 1) / splits;
  msplit = (msplit + kBM - 1) / kBM * kBM;
  if (gr && map) mreduce_act8_grouped_kernel<TJ, kPVec, true><<<grid, block, 0, st>>>(P, q, map, r, part, *gr);
  else if (gr) mreduce_act8_grouped_kernel<TJ, kPVec, false><<<grid, block, 0, st>>>(P, q, map, r, part, *gr);
  else mreduce_act8_kernel<TJ, kPVec><<<grid, block, 0, st>>>(P, q, M, r, msplit, part);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------- gate/up pair
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + __expf(-x)); }

// dYg = dH Yu silu'(Yg), dYu = dH silu(Yg), as in swiglu.hip, with Yg and Yu (2n columns a row) in 8 bits.
// A piece is 8 columns; n % 8 == 0, so that each lies in one block.
__global__ __launch_bounds__(256) void swiglu_bwd_act8_kernel(const uint16_t *__restrict__ dh, Act8 y, int64_t n,
                                                              uint16_t *__restrict__ dygu) {
  const int64_t pieces = n / 8, total = y.rows * pieces, nb = y.kp / kAct8Block;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / pieces, c = (i - row * pieces) * 8;
    const u32x4 d = *reinterpret_cast<const u32x4 *>(dh + row * n + c);
    const u32x2 g = *reinterpret_cast<const u32x2 *>(y.codes + row * y.kp + c);
    const u32x2 u = *reinterpret_cast<const u32x2 *>(y.codes + row * y.kp + n + c);
    const float sg = y.scale[row * nb + c / kAct8Block], su = y.scale[row * nb + (n + c) / kAct8Block];
    u32x4 og, ou;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float rg[2], ru[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float dv = h ? bf16_hi(d[e]) : bf16_lo(d[e]);
        const float gv = code_value(g[e >> 1], 2 * (e & 1) + h, sg);
        const float uv = code_value(u[e >> 1], 2 * (e & 1) + h, su);
        const float s = sigmoid(gv);
        rg[h] = dv * uv * (s * (1.f + gv * (1.f - s)));
        ru[h] = dv * (gv * s);
      }
      og[e] = pack_bf16x2(rg[0], rg[1]);
      ou[e] = pack_bf16x2(ru[0], ru[1]);
    }
    *reinterpret_cast<u32x4 *>(dygu + row * 2 * n + c) = og;
    *reinterpret_cast<u32x4 *>(dygu + row * 2 * n + n + c) = ou;
  }
}

bool vec_rows(const void *x, int64_t ldx, int64_t k, size_t esz) {
  return (((uintptr_t)x | (uintptr_t)(ldx * (int64_t)esz) | (uintptr_t)(k * (int64_t)esz)) & 15) == 0;
}

}  // namespace

hipError_t launch_act8_pack(const void *x, bool f32, int64_t ldx, const Act8 &q, hipStream_t st) {
  const int64_t blocks = (q.rows * (q.kp / 16) + 255) / 256;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 g((unsigned)blocks), b(256);
  const bool vec = vec_rows(x, ldx, q.k, f32 ? 4 : 2);
  if (f32) {
    if (vec) act8_pack_kernel<float, true><<<g, b, 0, st>>>((const float *)x, ldx, q);
    else act8_pack_kernel<float, false><<<g, b, 0, st>>>((const float *)x, ldx, q);
  } else {
    if (vec) act8_pack_kernel<uint16_t, true><<<g, b, 0, st>>>((const uint16_t *)x, ldx, q);
    else act8_pack_kernel<uint16_t, false><<<g, b, 0, st>>>((const uint16_t *)x, ldx, q);
  }
  return hipGetLastError();
}

hipError_t launch_act8_unpack(const Act8 &q, void *x, bool f32, int64_t ldx, hipStream_t st) {
  const int64_t blocks = (q.rows * (q.kp / 16) + 255) / 256;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 g((unsigned)blocks), b(256);
  const bool vec = vec_rows(x, ldx, q.k, f32 ? 4 : 2);
  if (f32) {
    if (vec) act8_unpack_kernel<float, true><<<g, b, 0, st>>>(q, (float *)x, ldx);
    else act8_unpack_kernel<float, false><<<g, b, 0, st>>>(q, (float *)x, ldx);
  } else {
    if (vec) act8_unpack_kernel<uint16_t, true><<<g, b, 0, st>>>(q, (uint16_t *)x, ldx);
    else act8_unpack_kernel<uint16_t, false><<<g, b, 0, st>>>(q, (uint16_t *)x, ldx);
  }
  return hipGetLastError();
}

// One round of workgroups, as many as the LDS of the 256 CUs holds (160 KB each; 16384 x 14336, rank 32, two a CU:
// 224 and 504 workgroups 73 and 67 us; 8192 x 4096, rank 64, one a CU: 256 and 512 workgroups 16.5 and 23 us).
int mreduce_act8_splits(int64_t M, int64_t C, int r, int E) {
  const int tj = (r + 15) / 16, nw = act8_waves(tj);
  const int lds = 2 * kBM * (32 * nw + 16) + 2 * (nw / 2) * kBM * (16 * tj + 8) * 2;
  const int64_t width = 32 * nw, tiles = (C + width - 1) / width * E;
  int64_t s = 256 * (160 * 1024 / lds < 2 ? 1 : 2) / tiles;
  const int64_t maxs = (M + kBM - 1) / kBM;
  s = s < maxs ? s : maxs;
  return (int)(s < 1 ? 1 : s);
}

hipError_t launch_mreduce_act8(const float *P, const Act8 &q, const int *map, int64_t M, int r, float s, int splits,
                               float *part, uint16_t *out, const GroupArgs *gr, hipStream_t st) {
  if (map && !gr) return hipErrorInvalidValue;
  hipError_t e = hipErrorInvalidValue;
  switch ((r + 15) / 16) {
#define MR_CASE(T)                                                                       \
  case T:                                                                                \
    e = (r & 3) ? launch_mreduce_act8_as<T, false>(P, q, map, M, r, splits, part, gr, st) \
                : launch_mreduce_act8_as<T, true>(P, q, map, M, r, splits, part, gr, st); \
    break;
    MR_CASE(1) MR_CASE(2) MR_CASE(3) MR_CASE(4) MR_CASE(5) MR_CASE(6) MR_CASE(7) MR_CASE(8)
#undef MR_CASE
    default: break;
  }
  if (e != hipSuccess) return e;
  return launch_mreduce_final(part, q.k, r, splits, gr ? gr->E : 1, s, false, out, st);
}

hipError_t launch_swiglu_bwd_act8(const uint16_t *dh, const Act8 &ygu, int64_t n, uint16_t *dygu, hipStream_t st) {
  if (n % 8) return hipErrorInvalidValue;
  int64_t b = (ygu.rows * n / 8 + 255) / 256;
  if (b > 8192) b = 8192;
  swiglu_bwd_act8_kernel<<<dim3((unsigned)(b < 1 ? 1 : b)), dim3(256), 0, st>>>(dh, ygu, n, dygu);
  return hipGetLastError();
}

}  // namespace nf4q
