// Backward pass of the output stage: the gradient by the logits back through
// soft cap, scale, the quantised matrix and the final norm.
//
// Per batch row b, with gl = dloss/dlogits and the forward's logits l:
//     t_v  = gl_v * scale * (cap > 0 ? (cap - l_v)(cap + l_v) / cap^2 : 1)
//     gx_k = sum_v t_v W_vk,     W_vk = d sc q - dmin m
// and with the norm, r = 1/sqrt(mean h^2 + eps), xh = h r, gg = gx gamma:
//     gh = r (gg - xh mean(gg xh)),   ggamma = sum_b gx xh
//
// Two launches: partial sums over a share of the rows of W for one block column
// (256 inputs), then their sum in a fixed order with the norm's backward.
#include "common.cuh"
#include "internal.h"

namespace muse {
namespace {

constexpr int kTileB = 8;        // batch rows a CTA holds sums of
constexpr int kShareRows = 64;   // rows of W whose t_v are staged at once

template <bool kQ4>
__global__ void __launch_bounds__(256) backward_kernel(const BackwardArgs a) {
  constexpr int kBB = kQ4 ? kBlockBytesQ4 : kBlockBytes;
  constexpr int kQs = kQ4 ? kOffQsQ4 : kOffQs;
  __shared__ float s_t[kShareRows][kTileB];
  const int nb = a.k / kBlockWeights;
  const int kb = blockIdx.x, part = blockIdx.y, b0 = blockIdx.z * kTileB;
  const int64_t lo = a.n_rows * part / gridDim.y, hi = a.n_rows * (part + 1) / gridDim.y;
  const int e = threadIdx.x, s = e >> 5, l = e & 31;
  float acc[kTileB] = {};
  for (int64_t v0 = lo; v0 < hi; v0 += kShareRows) {
    __syncthreads();
    for (int i = threadIdx.x; i < kShareRows * kTileB; i += 256) {
      const int b = i / kShareRows;
      const int64_t v = v0 + i % kShareRows;
      float t = 0.0f;
      if (v < hi && b0 + b < a.batch) {
        const int64_t at = static_cast<int64_t>(b0 + b) * a.n_rows + v;
        t = a.grad_logits[at] * a.scale;
        if (a.cap > 0.0f) t *= (a.cap - a.logits[at]) * (a.cap + a.logits[at]) / (a.cap * a.cap);
      }
      s_t[i % kShareRows][b] = t;
    }
    __syncthreads();
    for (int64_t v = v0; v < hi && v < v0 + kShareRows; ++v) {
      const uint8_t *blk = a.w + (v * nb + kb) * kBB;
      const uint4 hdr = __ldg(reinterpret_cast<const uint4 *>(blk));
      const float d = __half2float(__ushort_as_half(static_cast<unsigned short>(hdr.x & 0xFFFFu)));
      const float dmin = __half2float(__ushort_as_half(static_cast<unsigned short>(hdr.x >> 16)));
      int sc, mn;
      q5k_scale_min(hdr.y, hdr.z, hdr.w, s, sc, mn);
      int q = (blk[kQs + 32 * (s >> 1) + l] >> (4 * (s & 1))) & 15;
      if (!kQ4) q |= ((blk[kOffQh + l] >> s) & 1) << 4;
      const float w = fmaf(d * static_cast<float>(sc), static_cast<float>(q), -dmin * static_cast<float>(mn));
      for (int b = 0; b < kTileB; ++b) acc[b] = fmaf(s_t[v - v0][b], w, acc[b]);
    }
  }
  for (int b = 0; b < kTileB && b0 + b < a.batch; ++b)
    a.part[(static_cast<int64_t>(part) * a.batch + b0 + b) * a.k + kb * kBlockWeights + e] = acc[b];
}

// One CTA per batch row: gx = the parts' sum in order, then the norm's backward.
// gx stays in the first part's place for the gamma gradient.
__global__ void __launch_bounds__(256) backward_norm_kernel(const BackwardArgs a, int parts) {
  __shared__ float s_red[2][8];
  const int b = blockIdx.x;
  const int64_t stride = static_cast<int64_t>(a.batch) * a.k;
  float *gx = a.part + static_cast<int64_t>(b) * a.k;
  const float *h = a.hidden + static_cast<int64_t>(b) * a.k;
  float ss = 0.0f, dot = 0.0f;
  for (int j = threadIdx.x; j < a.k; j += 256) {
    float v = 0.0f;
    for (int p = 0; p < parts; ++p) v += gx[p * stride + j];
    gx[j] = v;
    if (a.gamma) {
      ss = fmaf(h[j], h[j], ss);
      dot = fmaf(v * a.gamma[j], h[j], dot);
    } else {
      a.grad_hidden[static_cast<int64_t>(b) * a.k + j] = v;
    }
  }
  if (!a.gamma) return;
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    dot += __shfl_xor_sync(0xffffffffu, dot, o);
  }
  if ((threadIdx.x & 31) == 0) {
    s_red[0][threadIdx.x >> 5] = ss;
    s_red[1][threadIdx.x >> 5] = dot;
  }
  __syncthreads();
  ss = dot = 0.0f;
  for (int i = 0; i < 8; ++i) {
    ss += s_red[0][i];
    dot += s_red[1][i];
  }
  const float r = 1.0f / sqrtf(ss / static_cast<float>(a.k) + a.eps);
  const float c = r * r * dot / static_cast<float>(a.k);
  if (threadIdx.x == 0) a.rms[b] = r;
  for (int j = threadIdx.x; j < a.k; j += 256)
    a.grad_hidden[static_cast<int64_t>(b) * a.k + j] = r * (gx[j] * a.gamma[j] - h[j] * c);
}

__global__ void __launch_bounds__(256) backward_gamma_kernel(const BackwardArgs a) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  float v = 0.0f;
  for (int b = 0; b < a.batch; ++b) {
    const int64_t at = static_cast<int64_t>(b) * a.k + j;
    v = fmaf(a.part[at] * a.rms[b], a.hidden[at], v);
  }
  a.grad_gamma[j] = v;
}

}  // namespace

constexpr int kBackwardParts = 12;

size_t backward_part_floats(int max_batch, int k) { return static_cast<size_t>(kBackwardParts) * max_batch * k; }

cudaError_t launch_backward(const BackwardArgs &a) {
  const int nb = a.k / kBlockWeights;
  const int parts = a.n_rows < kBackwardParts ? static_cast<int>(a.n_rows) : kBackwardParts;
  const dim3 grid(nb, parts, (a.batch + kTileB - 1) / kTileB);
  if (a.q4) backward_kernel<true><<<grid, 256, 0, a.stream>>>(a);
  else backward_kernel<false><<<grid, 256, 0, a.stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  backward_norm_kernel<<<a.batch, 256, 0, a.stream>>>(a, parts);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.grad_gamma) return e;
  backward_gamma_kernel<<<nb, 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace muse
