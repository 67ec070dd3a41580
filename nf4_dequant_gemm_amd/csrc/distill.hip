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
// takes a row and keeps it in registers (16 bytes a chunk, all of a thread's loads issued before the
// first is used), so that maximum, sum and gradient need no second read; a row longer than its
// registers is walked twice, with a running maximum and sum, and comes from the caches the second
// time. Sums and statistics are float32; the gradient is rounded once. Rows need not be aligned: the
// few elements before the first and after the last 16-byte boundary are taken one by one.
// Gradient entries of the teacher's indices are written after the others, by one thread for each
// distinct index, so that the result does not depend on any order.
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

template <int kThreads>
struct Red {
  float v[kThreads / 64];
  // Maximum / sum over the workgroup, the same in every thread (waves in order).
  __device__ __forceinline__ float max(float x) {
    for (int o = 32; o; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
    return meet(x, true);
  }
  __device__ __forceinline__ float sum(float x) {
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    return meet(x, false);
  }
  __device__ __forceinline__ float meet(float x, bool is_max) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) v[threadIdx.x >> 6] = x;
    __syncthreads();
    x = v[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) x = is_max ? fmaxf(x, v[w]) : x + v[w];
    return x;
  }
};

// kChunks chunks a thread: the row stays in registers. kChunks 0: the row is walked twice.
template <typename XT, int kThreads, int kChunks>
__global__ __launch_bounds__(kThreads) void distill_kernel(DistillArgs a) {
  constexpr int P = kPer<XT>;
  __shared__ Red<kThreads> red;
  __shared__ int s_idx[kDistillMaxTop];
  __shared__ float s_p[kDistillMaxTop];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const XT *z = reinterpret_cast<const XT *>(a.z) + row * a.ld;
  XT *dz = a.dz ? reinterpret_cast<XT *>(a.dz) + row * a.ldd : nullptr;
  const float w = dz && a.weight ? a.weight[row] : 1.f;
  const float c2 = kLog2e / a.tau;
  const int v = (int)a.v, top = a.top;
  // chunks: [0, head) one by one, then n chunks, then [tail, v) one by one; the gradient's rows
  // must lie as the logits' do for its chunks to be whole (else they are stored one by one)
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
      reinterpret_cast<u32x4 *>(dz + head)[i] = o;
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) dz[head + i * P + e] = from_f32<XT>(y[e]);
    }
  };

  if (w == 0.f) {   // workgroup-uniform: nothing of the row is read
    if (tid == 0) {
      if (a.loss) a.loss[row] = 0.f;
      if (a.lse) a.lse[row] = 0.f;
    }
    const float zero[P] = {};
    for (int i = tid; i < n; i += kThreads) put_chunk(i, zero);
    if (odd >= 0) dz[odd] = from_f32<XT>(0.f);
    return;
  }

  // ---- the row's maximum and sum of exp2((z - max) c2)
  constexpr int NC = kChunks > 0 ? kChunks : 1;
  u32x4 c[NC];
  float zo = -INFINITY, top_z = -INFINITY, sum = 0.f;
  if (kChunks > 0) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int i = tid + j * kThreads;
      if (i < n) c[j] = zc[i];
    }
  }
  if (odd >= 0) zo = to_f32<XT>(z[odd]);
  // the teacher's entries: index, logit and the student's logit there (before dz may overwrite it)
  constexpr int kMine = (kDistillMaxTop + kThreads - 1) / kThreads;
  int ti[kMine];
  float ty[kMine], tz[kMine];
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
  }
  float ln_sum = 0.f;                       // log2 of the sum
  if (!a.lse_in) {
    if (kChunks > 0) {
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (tid + j * kThreads < n)
#pragma unroll
          for (int e = 0; e < P; ++e) top_z = fmaxf(top_z, elem<XT>(c[j], e));
      top_z = red.max(fmaxf(top_z, zo));
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (tid + j * kThreads < n)
#pragma unroll
          for (int e = 0; e < P; ++e) sum += __builtin_amdgcn_exp2f((elem<XT>(c[j], e) - top_z) * c2);
    } else {
      // running maximum m and sum over batches of four chunks
      float m = zo;
      float s = 0.f;
      for (int i0 = tid; i0 < n; i0 += 4 * kThreads) {
        u32x4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + j * kThreads < n) b[j] = zc[i0 + j * kThreads];
        float bm = m;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + j * kThreads < n)
#pragma unroll
            for (int e = 0; e < P; ++e) bm = fmaxf(bm, elem<XT>(b[j], e));
        if (bm > m) {
          s *= __builtin_amdgcn_exp2f((m - bm) * c2);   // m = -inf: s is 0, exp2(-inf) = 0
          m = bm;
        }
        if (m > -INFINITY) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i0 + j * kThreads < n)
#pragma unroll
              for (int e = 0; e < P; ++e) s += __builtin_amdgcn_exp2f((elem<XT>(b[j], e) - m) * c2);
        }
      }
      top_z = red.max(m);
      if (m > -INFINITY) sum = s * __builtin_amdgcn_exp2f((m - top_z) * c2);
    }
    if (odd >= 0) sum += __builtin_amdgcn_exp2f((zo - top_z) * c2);
    sum = red.sum(sum);
    ln_sum = __builtin_amdgcn_logf(sum);    // base 2
  } else {
    // lse / tau known: (z - 0) c2 - lse log2(e)
    top_z = 0.f;
    ln_sum = a.lse_in[row] * kLog2e;
  }

  // ---- the teacher's distribution
  float my = -INFINITY;
#pragma unroll
  for (int q = 0; q < kMine; ++q) my = fmaxf(my, ty[q] != ty[q] ? INFINITY : ty[q]);   // a NaN makes the row NaN
  my = red.max(my);
  float ps = 0.f;
  const bool any = my > -INFINITY;
#pragma unroll
  for (int q = 0; q < kMine; ++q)
    if (any && ti[q] >= 0) ps += expf((ty[q] - my) / a.tau);
  ps = red.sum(ps);
  const float log_ps = logf(ps);
  float part = 0.f;
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int k = tid + q * kThreads;
    float p = 0.f;
    if (any && ti[q] >= 0) {
      const float lp = (ty[q] - my) / a.tau - log_ps;
      p = expf(lp);
      // log q = (z - max) / tau - ln(sum)
      if (p > 0.f || p != p) part += p * (lp - ((tz[q] - top_z) / a.tau - ln_sum * kLn2));
    }
    if (k < top) {
      s_idx[k] = p == 0.f ? -1 : ti[q];
      s_p[k] = p;
    }
  }
  if (a.loss) {
    part = red.sum(part);
    if (tid == 0) a.loss[row] = part;
  }
  if (a.lse && tid == 0) a.lse[row] = top_z / a.tau + ln_sum * kLn2;
  if (!dz) return;

  // ---- the gradient
  const float wt = w / a.tau;
  if (!any) {   // no entries: zero (workgroup-uniform)
    const float zero[P] = {};
    for (int i = tid; i < n; i += kThreads) put_chunk(i, zero);
    if (odd >= 0) dz[odd] = from_f32<XT>(0.f);
    return;
  }
  __syncthreads();   // s_idx, s_p; and every gathered logit is in registers before dz = z is written
  auto grad = [&](float x) { return wt * __builtin_amdgcn_exp2f((x - top_z) * c2 - ln_sum); };
  if (kChunks > 0) {
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
    float p = 0.f;
    bool first = true;
    for (int o = 0; o < top; ++o) {
      const bool eq = s_idx[o] == i;
      first = first && !(eq && o < k);
      p += eq ? s_p[o] : 0.f;
    }
    if (first) dz[i] = from_f32<XT>(wt * (__builtin_amdgcn_exp2f((tz[q] - top_z) * c2 - ln_sum) - p));
  }
}

template <typename XT>
hipError_t launch_type(const DistillArgs &a, hipStream_t st) {
  const int64_t chunks = a.v / kPer<XT> + 1;
  const dim3 grid((unsigned)a.t);
  if (chunks <= 256 * 8)
    distill_kernel<XT, 256, 8><<<grid, dim3(256), 0, st>>>(a);
  else if (chunks <= 1024 * 8)
    distill_kernel<XT, 1024, 8><<<grid, dim3(1024), 0, st>>>(a);
  else if (chunks <= 1024 * 16)
    distill_kernel<XT, 1024, 16><<<grid, dim3(1024), 0, st>>>(a);
  else
    distill_kernel<XT, 1024, 0><<<grid, dim3(1024), 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_distill(const DistillArgs &a, bool f32, hipStream_t st) {
  if (a.t < 1 || a.t >= (int64_t(1) << 31) || a.v < 1 || a.v >= (int64_t(1) << 30) || a.top < 1 || a.top > kDistillMaxTop)
    return hipErrorInvalidValue;
  return f32 ? launch_type<float>(a, st) : launch_type<uint16_t>(a, st);
}

}  // namespace nf4q
