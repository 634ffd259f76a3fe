// Distillation from a teacher's top alternatives: each row's loss and its
// gradient by the student's logits.
//
// Student row x of V logits, z = x / T, q = softmax(z).  Teacher entries
// (id_j, l_j), those with an id outside 0..V-1 left out, S the set of ids:
//     renormalised: p_j = exp(l_j) / sum exp(l),  p_t = 0
//     tail:         p_j = exp(l_j),  p_t = max(0, 1 - sum p),  q_t = sum_{i not in S} q_i
//     loss = w [ sum_j p_j (log p_j - log q_{id_j}) + p_t (log p_t - log q_t) ]
//     dloss/dx_i = w/T [ (sum p + p_t) q_i - sum_{j: id_j = i} p_j - [i not in S] p_t q_i / q_t ]
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kDistillThreads = 512;

__device__ __forceinline__ float block_sum(float v, float *s) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.0f;
  for (int w = 0; w < kDistillThreads / 32; ++w) r += s[w];
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kDistillThreads) distill_kernel(const DistillArgs a) {
  __shared__ float s_red[kDistillThreads / 32];
  __shared__ float s_max[kDistillThreads / 32];
  __shared__ int s_id[kMaxTop];
  __shared__ float s_x[kMaxTop], s_p[kMaxTop];
  __shared__ uint32_t s_seen[64];                      // 2,048 bits: ids mod 2,048
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  T *g = a.grad ? static_cast<T *>(a.grad) + row * a.grad_ld : nullptr;
  const int v = static_cast<int>(a.v), tid = threadIdx.x;
  const float inv_t = 1.0f / a.temperature;
  const float w = a.row_weight ? a.row_weight[row] : 1.0f;

  if (tid < 64) s_seen[tid] = 0u;
  float m = -INFINITY;
  for (int i = tid; i < v; i += kDistillThreads) m = fmaxf(m, to_float(x[i]));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
  for (int i = 0; i < kDistillThreads / 32; ++i) m = fmaxf(m, s_max[i]);
  if (tid < a.n_top) {
    const int id = a.teacher_ids[row * a.n_top + tid];
    const bool ok = id >= 0 && id < v;
    s_id[tid] = ok ? id : -1;
    s_p[tid] = ok ? a.teacher_logprobs[row * a.n_top + tid] : -INFINITY;
    s_x[tid] = ok ? to_float(x[id]) : 0.0f;
    if (ok) atomicOr(&s_seen[(id & 2047) >> 5], 1u << (id & 31));
  }
  __syncthreads();
  if (m == -INFINITY) m = 0.0f;        // all masked (the sum stays 0), or NaN beside masked values (it turns NaN)
  auto named = [&](int i) {
    if (!((s_seen[(i & 2047) >> 5] >> (i & 31)) & 1u)) return false;
    for (int j = 0; j < a.n_top; ++j)
      if (s_id[j] == i) return true;
    return false;
  };
  float rest = 0.0f, in = 0.0f;
  for (int i = tid; i < v; i += kDistillThreads) {
    const float e = expf((to_float(x[i]) - m) * inv_t);
    if (named(i)) in += e;
    else rest += e;
  }
  rest = block_sum(rest, s_red);
  in = block_sum(in, s_red);
  const float total = rest + in, logs = logf(total);
  if (w == 0.0f || total == 0.0f) {                    // no weight, or a row without a distribution
    if (tid == 0 && a.loss) a.loss[row] = 0.0f;
    if (g)
      for (int i = tid; i < v; i += kDistillThreads) g[i] = from_float<T>(0.0f);
    return;
  }

  float lmax = -INFINITY, mass = 0.0f, loss = 0.0f;
  for (int j = 0; j < a.n_top; ++j) lmax = fmaxf(lmax, s_p[j]);
  if (lmax > -INFINITY) {
    float sum = 0.0f;
    for (int j = 0; j < a.n_top; ++j) sum += expf(s_p[j] - lmax);
    const float c = a.tail ? 0.0f : lmax + logf(sum);
    for (int j = 0; j < a.n_top; ++j) {
      const float lp = s_p[j] - c, p = expf(lp);
      mass += p;
      if (p > 0.0f) loss += p * (lp - ((s_x[j] - m) * inv_t - logs));
    }
    __syncthreads();
    if (tid < a.n_top) s_p[tid] = expf(s_p[tid] - c);
  } else {
    __syncthreads();
    if (tid < a.n_top) s_p[tid] = 0.0f;
  }
  const float pt = a.tail ? fmaxf(0.0f, 1.0f - mass) : 0.0f;
  if (pt > 0.0f) loss += pt * (logf(pt) - (logf(rest) - logs));
  if (tid == 0 && a.loss) a.loss[row] = w * loss;
  if (!g) return;
  __syncthreads();
  const float scale = w * inv_t;
  const float f_in = (mass + pt) / total * scale;
  const float f_out = rest != 0.0f ? ((mass + pt) / total - pt / rest) * scale : 0.0f;
  for (int i = tid; i < v; i += kDistillThreads) {
    const float e = expf((to_float(x[i]) - m) * inv_t);
    float r = e * f_out;
    if (named(i)) {
      r = e * f_in;
      for (int j = 0; j < a.n_top; ++j)
        if (s_id[j] == i) r -= s_p[j] * scale;
    }
    g[i] = from_float<T>(r);
  }
}

}  // namespace

cudaError_t launch_distill(const DistillArgs &a) {
  const unsigned grid = static_cast<unsigned>(a.n);
  if (a.dtype == 0) distill_kernel<float><<<grid, kDistillThreads, 0, a.stream>>>(a);
  else if (a.dtype == 1) distill_kernel<__half><<<grid, kDistillThreads, 0, a.stream>>>(a);
  else distill_kernel<__nv_bfloat16><<<grid, kDistillThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace muse
