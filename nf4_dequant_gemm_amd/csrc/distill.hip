// Distillation loss from a teacher's top logits, and its gradient (gfx950).
//
// For one row z[0 .. v) of student logits, the teacher's kept entries (idx_k, y_k), k < top, and a
// temperature tau:
//
//   log q_i = z_i / tau - lse,  lse = log sum_i exp(z_i / tau)
//   p       = softmax of y_k / tau over the kept entries
//   loss    = sum_k p_k (log p_k - log q[idx_k]),   dz_i = (w / tau) (q_i - sum_{k: idx_k = i} p_k)
//
// with w the row's weight. An entry whose index lies outside [0, v) or whose teacher logit is -inf
// is not there; a row without entries has loss 0 and gradient 0, and so has a row of weight 0,
// which is not read.
//
// The work is one read of the logits and, with the gradient, one write: memory bound. A workgroup
// takes a row. With the gradient it keeps the row in registers (16 bytes a chunk, all of a thread's loads
// issued before the first is used), so that maximum, sum and gradient need no second read; a row longer
// than that, and a row whose gradient is not wanted or whose lse is known, is walked with a running
// maximum and sum, for the gradient a second time (from the caches; with a known lse that time only:
// 4096 x 128000 399 us, 1024 x 50001 in float32 90 us). Two exchanges over the workgroup are
// enough, since with u_k = exp((y_k - max y) / tau)
//
//   loss = sum_k u_k ((y_k - max y) - (z[idx_k] - max z)) / tau / sum u - log sum u + log sum exp((z - max z) / tau):
//
// the two maxima, then the three sums together. Sums and statistics are float32; the gradient is rounded
// once and streamed out (non-temporal: 523 -> 472 us on 4096 x 128000). Rows need not be aligned: the
// few elements before the first and after the last 16-byte boundary are taken one by one. Gradient
// entries of the teacher's indices are written after the others, by one thread for each distinct index,
// so that the result does not depend on any order.
#include "common.h"
#include "launch.h"

namespace nf4q {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

template <typename XT>
__device__ __forceinline__ float to_f32(XT v);
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <typename XT>
__device__ __forceinline__ XT from_f32(float v);
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// Elements of a 16-byte chunk and element e of it.
template <typename XT>
constexpr int kPer = 16 / (int)sizeof(XT);
template <typename XT>
__device__ __forceinline__ float elem(const u32x4 &c, int e) {
  if constexpr (sizeof(XT) == 2) {
    return (e & 1) ? bf16_hi(c[e >> 1]) : bf16_lo(c[e >> 1]);
  } else {
    return __uint_as_float(c[e]);
  }
}

// kThreads threads a row. kChunks chunks a thread: the row stays in registers; 0: it is walked. At most
// kTop<kThreads> entries of the teacher.
template <int kThreads>
constexpr int kTop = 4 * kThreads < kDistillMaxTop ? 4 * kThreads : kDistillMaxTop;

// Waves a SIMD: what the row's registers allow. Left to itself the compiler unpacks a whole float32 row of
// 8 chunks at once (244 registers, 92 us instead of 50 on 2048 x 16000).
template <typename XT, int kThreads, int kChunks>
__global__ __launch_bounds__(kThreads, kChunks <= 8 ? 6 : 4) void distill_kernel(DistillArgs a) {
  constexpr int P = kPer<XT>, kWaves = kThreads / 64;
  __shared__ float s_max[2][kWaves], s_sum[3][kWaves];
  __shared__ __align__(16) int s_idx[kTop<kThreads>];
  __shared__ float s_u[kTop<kThreads>];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.t) return;
  const XT *z = reinterpret_cast<const XT *>(a.z) + row * a.ld;
  XT *dz = a.dz ? reinterpret_cast<XT *>(a.dz) + row * a.ldd : nullptr;
  const float w = dz && a.weight ? a.weight[row] : 1.f;
  const float c2 = kLog2e / a.tau;
  const int v = (int)a.v, top = a.top;
  // elements [0, head) one by one, then n chunks, then [tail, v) one by one; a gradient whose row does not
  // lie as the logits' does is stored one by one throughout
  const int mis = (int)((reinterpret_cast<uintptr_t>(z) / sizeof(XT)) % P);
  int head = mis ? P - mis : 0;
  head = head < v ? head : v;
  const int n = (v - head) / P;
  const int tail = head + n * P;
  const u32x4 *zc = reinterpret_cast<const u32x4 *>(z + head);
  const bool same = dz && ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
  // the odd element of this thread, if any: head elements by threads 0 .. P - 1, tail by P .. 2 P - 1
  const int odd = tid < P ? (tid < head ? tid : -1)
                          : (tid < 2 * P && tail + tid - P < v ? tail + tid - P : -1);

  auto put_chunk = [&](int i, const float *y) {
    if (same) {
      u32x4 o;
      if constexpr (P == 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(y[2 * e], y[2 * e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(y[e]);
      }
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4 *>(dz + head) + i);
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) dz[head + i * P + e] = from_f32<XT>(y[e]);
    }
  };
  auto put_zeros = [&]() {
    const float zero[P] = {};
    for (int i = tid; i < n; i += kThreads) put_chunk(i, zero);
    if (odd >= 0) dz[odd] = from_f32<XT>(0.f);
  };

  if (w == 0.f) {   // the whole workgroup: nothing of the row is read
    if (tid == 0) {
      if (a.loss) a.loss[row] = 0.f;
      if (a.lse) a.lse[row] = 0.f;
    }
    put_zeros();
    return;
  }

  // ---- the teacher's entries: index, logit and the student's logit there (before dz may overwrite it)
  constexpr int NC = kChunks > 0 ? kChunks : 1;
  u32x4 c[NC];
  if constexpr (kChunks > 0) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int i = tid + j * kThreads;
      if (i < n) c[j] = zc[i];
    }
  }
  const float zo = odd >= 0 ? to_f32<XT>(z[odd]) : -INFINITY;
  constexpr int kMine = kTop<kThreads> / kThreads;
  int ti[kMine];
  float ty[kMine], tz[kMine];
  float my = -INFINITY;
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int k = tid + q * kThreads;
    ti[q] = -1;
    ty[q] = -INFINITY;
    tz[q] = 0.f;
    if (k < top) {
      const int i = a.idx[row * top + k];
      if (i >= 0 && i < v) {
        ti[q] = i;
        ty[q] = a.teacher[row * top + k];
        tz[q] = to_f32<XT>(z[i]);
      }
    }
    my = fmaxf(my, ty[q] != ty[q] ? INFINITY : ty[q]);   // a NaN makes the row NaN
  }

  // ---- the maxima
  float top_z = zo, s = 0.f;   // this thread's running maximum, and its sum relative to it
  // A large lse has lost the digits of the sum (in a row masked with -1e9 throughout, log v of it) or has
  // overflowed: such a row's sum is formed again. Below 256 lse is off by at most 2^-17.
  const bool known = a.lse_in && fabsf(a.lse_in[row]) < 256.f;
  // four chunks (i0 + j kThreads, those below n) into the running maximum and sum
  auto take = [&](const u32x4 *b, int i0) {
    float m = top_z;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * kThreads < n)
#pragma unroll
        for (int e = 0; e < P; ++e) m = fmaxf(m, elem<XT>(b[j], e));
    if (m > top_z) {
      s *= __builtin_amdgcn_exp2f((top_z - m) * c2);   // from -inf: s is 0 or NaN, exp2(-inf) = 0
      top_z = m;
    }
    // The maximum passes over a NaN, so the sum takes every element whatever the maximum is: against 0
    // while that is -inf, exp2(-inf) = 0 for the masked ones and NaN for a NaN.
    const float ref = m > -INFINITY ? m : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * kThreads < n)
#pragma unroll
        for (int e = 0; e < P; ++e) s += __builtin_amdgcn_exp2f((elem<XT>(b[j], e) - ref) * c2);
  };
  if (!known) {
    if constexpr (kChunks > 0) {
#pragma unroll
      for (int j = 0; j < NC; j += 4) take(c + j, tid + j * kThreads);
    } else {
      for (int i0 = tid; i0 < n; i0 += 4 * kThreads) {
        u32x4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + j * kThreads < n) b[j] = zc[i0 + j * kThreads];
        take(b, i0);
      }
    }
  }
  const float mine = top_z;
  for (int o = 32; o; o >>= 1) {
    top_z = fmaxf(top_z, __shfl_xor(top_z, o));
    my = fmaxf(my, __shfl_xor(my, o));
  }
  if (lane == 0) {
    s_max[0][wave] = top_z;
    s_max[1][wave] = my;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kWaves; ++q) {
    top_z = fmaxf(top_z, s_max[0][q]);
    my = fmaxf(my, s_max[1][q]);
  }
  if (known) top_z = 0.f;
  const bool any = my > -INFINITY;   // the row has entries

  // ---- the sums: exp2((z - max) c2), u_k, u_k times the difference of the logs
  float sum = 0.f, us = 0.f, ds = 0.f;
  if (!known) {
    // of -inf alone, or with NaN: s is 0, or NaN, which stays
    sum = mine > -INFINITY ? s * __builtin_amdgcn_exp2f((mine - top_z) * c2) : s;
    if (odd >= 0) sum += __builtin_amdgcn_exp2f((zo - top_z) * c2);
  }
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int k = tid + q * kThreads;
    float u = 0.f;
    if (any && ti[q] >= 0) {
      const float ly = (ty[q] - my) / a.tau;
      u = expf(ly);
      us += u;
      if (u > 0.f || u != u) ds += u * (ly - (tz[q] - top_z) / a.tau);
    }
    if (k < kTop<kThreads>) {
      s_idx[k] = u == 0.f ? -1 : ti[q];
      s_u[k] = u;
    }
  }
  for (int o = 32; o; o >>= 1) {
    sum += __shfl_xor(sum, o);
    us += __shfl_xor(us, o);
    ds += __shfl_xor(ds, o);
  }
  if (lane == 0) {
    s_sum[0][wave] = sum;
    s_sum[1][wave] = us;
    s_sum[2][wave] = ds;
  }
  __syncthreads();   // also: every gathered logit is in registers before dz = z may be written
  sum = us = ds = 0.f;
#pragma unroll
  for (int q = 0; q < kWaves; ++q) {
    sum += s_sum[0][q];
    us += s_sum[1][q];
    ds += s_sum[2][q];
  }
  // log2 of the sum; with lse known, that of exp2(lse log2 e) against a maximum of 0
  const float l2 = known ? a.lse_in[row] * kLog2e : __builtin_amdgcn_logf(sum);
  if (tid == 0) {
    if (a.loss) a.loss[row] = any ? ds / us - logf(us) + l2 * kLn2 : 0.f;
    if (a.lse) a.lse[row] = top_z / a.tau + l2 * kLn2;
  }
  if (!dz) return;
  if (!any) {   // the whole workgroup
    put_zeros();
    return;
  }

  // ---- the gradient
  const float wt = w / a.tau;
  auto grad = [&](float x) { return wt * __builtin_amdgcn_exp2f((x - top_z) * c2 - l2); };
  if constexpr (kChunks > 0) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int i = tid + j * kThreads;
      if (i < n) {
        float y[P];
#pragma unroll
        for (int e = 0; e < P; ++e) y[e] = grad(elem<XT>(c[j], e));
        put_chunk(i, y);
      }
    }
  } else {
    for (int i0 = tid; i0 < n; i0 += 4 * kThreads) {
      u32x4 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j * kThreads < n) b[j] = zc[i0 + j * kThreads];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j * kThreads < n) {
          float y[P];
#pragma unroll
          for (int e = 0; e < P; ++e) y[e] = grad(elem<XT>(b[j], e));
          put_chunk(i0 + j * kThreads, y);
        }
    }
  }
  if (odd >= 0) dz[odd] = from_f32<XT>(grad(zo));
  // the teacher's indices: the first entry of each distinct index writes q - (sum of its p). The
  // barrier orders these stores after the workgroup's others to the same places.
  __threadfence_block();
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int k = tid + q * kThreads;
    if (k >= top) continue;
    const int i = s_idx[k];
    if (i < 0) continue;
    // entries of the same index, four at a time (the list is padded with -1)
    int before = 0, all = 0;
    for (int o = 0; o < top; o += 4) {
      const int4 x = *reinterpret_cast<const int4 *>(s_idx + o);
      const int eq = (x.x == i) + (x.y == i) + (x.z == i) + (x.w == i);
      all += eq;
      before += o + 4 <= k ? eq : (x.x == i && o < k) + (x.y == i && o + 1 < k) + (x.z == i && o + 2 < k);
    }
    if (before) continue;
    float u = s_u[k];
    if (all > 1)
      for (int o = k + 1; o < top; ++o) u += s_idx[o] == i ? s_u[o] : 0.f;
    dz[i] = from_f32<XT>(wt * (__builtin_amdgcn_exp2f((tz[q] - top_z) * c2 - l2) - u / us));
  }
}

constexpr int64_t kGridRows = int64_t(1) << 21;
template <typename XT, int kThreads, int kChunks>
hipError_t launch_row(const DistillArgs &a, hipStream_t st) {
  // Fewer than 2^32 threads along a dimension: 67 million rows of 64 threads in one were taken modulo that,
  // without an error, and left all but the first few rows unwritten.
  const int64_t x = a.t < kGridRows ? a.t : kGridRows;
  const dim3 grid((unsigned)x, (unsigned)((a.t + x - 1) / x));
  distill_kernel<XT, kThreads, kChunks><<<grid, dim3(kThreads), 0, st>>>(a);
  return hipGetLastError();
}

// Threads a row, by its 16-byte chunks: the fewest that hold it in registers with 8 (16) chunks each, since
// several small workgroups on a CU overlap their loads and their arithmetic (4096 x 32000 in bf16 with the
// gradient: 256 threads of 16 chunks 110 us, 512 of 8 106 us, 1024 of 4 132 us, walked by 512 122 us); past
// 512 of 16, walked by 1024 (4096 x 128000: 451 us, 512 of 32 489 us, 1024 of 16 472 us). Without the
// gradient nothing need stay: walked (1024 x 50001 in float32: 38 us, in registers 56 us). The sum runs
// over the same chunks in the same order either way, so the loss alone and the loss with the gradient
// agree bit for bit. 64-thread workgroups need no more than 256 entries.
template <typename XT>
hipError_t launch_type(const DistillArgs &a, hipStream_t st) {
  const int64_t chunks = a.v / kPer<XT> + 1;
  if (chunks <= 64 * 8 && a.top <= kTop<64>) return launch_row<XT, 64, 8>(a, st);
  if (a.dz && !a.lse_in) {
    if (chunks <= 256 * 4) return launch_row<XT, 256, 4>(a, st);
    if (chunks <= 256 * 8) return launch_row<XT, 256, 8>(a, st);
    if (chunks <= 512 * 8) return launch_row<XT, 512, 8>(a, st);
    if (chunks <= 512 * 16) return launch_row<XT, 512, 16>(a, st);
    return launch_row<XT, 1024, 0>(a, st);
  }
  if (chunks <= 256 * 8) return launch_row<XT, 256, 0>(a, st);
  if (chunks <= 512 * 16) return launch_row<XT, 512, 0>(a, st);
  return launch_row<XT, 1024, 0>(a, st);
}

}  // namespace

hipError_t launch_distill(const DistillArgs &a, bool f32, hipStream_t st) {
  if (a.t < 1 || a.t >= (int64_t(1) << 31) || a.v < 1 || a.v >= (int64_t(1) << 30) || a.top < 1 || a.top > kDistillMaxTop)
    return hipErrorInvalidValue;
  return f32 ? launch_type<float>(a, st) : launch_type<uint16_t>(a, st);
}

}  // namespace nf4q
