// Scores of finished logits: the log probability and rank of a given token,
// the normaliser, the entropy and the top alternatives of each row.
//
// For a row x of V logits, z = x / temperature and m = max z:
//     S = sum_i exp(z_i - m),  U = sum_i exp(z_i - m) (z_i - m)
//     lse = m + log S,  logprob(t) = z_t - lse,  entropy = log S - U / S
// Ranks and alternatives order by (x descending, index ascending), on x itself:
// a division could merge neighbouring values.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kScoreThreads = 512;

__device__ __forceinline__ float block_sum(float v, float *s) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.0f;
  for (int w = 0; w < kScoreThreads / 32; ++w) r += s[w];
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const ScoreArgs a) {
  __shared__ float s_red[kScoreThreads / 32];
  __shared__ unsigned long long s_key;
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  const int v = static_cast<int>(a.v);
  const float inv_t = 1.0f / a.temperature;

  float m = -INFINITY;
  for (int i = threadIdx.x; i < v; i += kScoreThreads) m = fmaxf(m, to_float(x[i]));
  if (threadIdx.x == 0) s_key = 0ull;
  __syncthreads();
  atomicMax(&s_key, argmax_key(m, 0u));
  __syncthreads();
  m = order_key_float(static_cast<uint32_t>(s_key >> 32));
  if (m == -INFINITY) m = 0.0f;       // all masked (the sum stays 0), or NaN beside masked values (it turns NaN)

  const int64_t tok = a.tokens ? a.tokens[row] : -1;
  const bool has = tok >= 0 && tok < v;
  const float xt = has ? to_float(x[tok]) : 0.0f;
  float s = 0.0f, u = 0.0f;
  int before = 0;
  for (int i = threadIdx.x; i < v; i += kScoreThreads) {
    const float xi = to_float(x[i]);
    const float dz = (xi - m) * inv_t;
    const float e = expf(dz);
    s += e;
    u += e > 0.0f ? e * dz : 0.0f;
    before += xi > xt || (xi == xt && i < tok);
  }
  s = block_sum(s, s_red);
  u = block_sum(u, s_red);
  before = static_cast<int>(block_sum(static_cast<float>(before), s_red));
  const bool empty = s == 0.0f;
  const float logs = logf(s), z0 = m * inv_t;
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[row] = empty ? -INFINITY : z0 + logs;
    if (a.entropy) a.entropy[row] = empty ? 0.0f : logs - u / s;
    if (a.logprob) a.logprob[row] = !has ? 0.0f : empty ? -INFINITY : (xt - m) * inv_t - logs;
    if (a.rank) a.rank[row] = has ? before : -1;
  }
  // alternatives: the largest key below the last one found, n_top times
  unsigned long long last = ~0ull;
  for (int j = 0; j < a.n_top; ++j) {
    __syncthreads();
    if (threadIdx.x == 0) s_key = 0ull;
    __syncthreads();
    unsigned long long best = 0ull;
    for (int i = threadIdx.x; i < v; i += kScoreThreads) {
      const unsigned long long key = argmax_key(to_float(x[i]), static_cast<uint32_t>(i));
      if (key < last && key > best) best = key;
    }
    if (best) atomicMax(&s_key, best);
    __syncthreads();
    last = s_key;
    if (threadIdx.x == 0) {
      const float xv = order_key_float(static_cast<uint32_t>(last >> 32));
      a.top_ids[row * a.n_top + j] = last ? static_cast<int32_t>(argmax_key_index(last)) : -1;
      a.top_logprobs[row * a.n_top + j] = !last || empty ? -INFINITY : (xv - m) * inv_t - logs;
    }
  }
}

}  // namespace

cudaError_t launch_score(const ScoreArgs &a) {
  const unsigned grid = static_cast<unsigned>(a.n);
  if (a.dtype == 0) score_kernel<float><<<grid, kScoreThreads, 0, a.stream>>>(a);
  else if (a.dtype == 1) score_kernel<__half><<<grid, kScoreThreads, 0, a.stream>>>(a);
  else score_kernel<__nv_bfloat16><<<grid, kScoreThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace muse
