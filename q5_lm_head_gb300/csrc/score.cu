// Scores of finished logits: the log probability and rank of a given token,
// the normaliser, the entropy and the top alternatives of each row.
//
// For a row x of V logits, z = x / temperature and m = max x:
//     a_i = (x_i - m) log2(e) / temperature,  S = sum_i 2^a_i,  U = sum_i 2^a_i a_i
//     lse = m / temperature + log S,  logprob(t) = (x_t - m) / temperature - log S,
//     entropy = log S - ln 2 U / S
// Ranks and alternatives order by (x descending, index ascending), on x itself:
// a division could merge neighbouring values.
//
// Bound: HBM (each logit is read once) for many rows, latency for a few.  A
// cluster of 1, 2, 4, 8 or 16 CTAs takes a row (as many as keep the GPU's CTA
// slots filled once), each a contiguous share of its 16-byte vectors; its
// threads hold a running maximum with S and U, and the CTAs' results meet in
// the first one's hands through distributed shared memory.  No global
// workspace, so calls may overlap.
//
// Alternatives: a thread's running maximum stands for one element of its own,
// so the n_top-th largest of the 512 maxima is a value that at least n_top
// elements reach.  Elements above that bound go to a list in shared memory; the
// bound is taken after the first step, on values still in registers, and again
// after 1, 2, 4, 8 .. steps, so a row lists about n_top log2(steps) elements.
// The bound's equals are not listed (a masked row would be nothing else): where
// fewer than n_top lie above it, the rest are its first equals by index, found
// by a scan that stops early.  A row whose list overflows (values rising along
// the row) takes the bound from bitwise counts over the row instead.
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 2048;              // listed elements, at least kMaxTop for each CTA of a cluster
constexpr int kMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;   // float_order_key(-infinity): below it only NaNs

// Maximum with the sums S and U against it; m = -infinity: nothing above -infinity seen
// (S and U are then 0, or NaN).
struct Stat {
  float m, s, u;
};

__device__ __forceinline__ Stat stat_join(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, a.s + b.s, a.u + b.u};
  auto move = [&](Stat &t) {             // onto the reference m
    const float d = (t.m - m) * c, f = exp2_approx(d);
    t.u = t.s == 0.0f ? 0.0f : (t.u + t.s * fmaxf(d, -1e30f)) * f;
    t.s *= f;
    if (t.m == -INFINITY) t.s = t.u = t.s != t.s ? t.s : 0.0f;
  };
  move(a);
  move(b);
  return {m, a.s + b.s, a.u + b.u};
}

struct Shared {
  unsigned long long list[kList];
  unsigned long long best[kMaxTop];
  float m[kWarps], s[kWarps], u[kWarps];
  int before[kWarps];
  uint32_t low[kWarps];
  int cnt[2][kWarps];
  float out_m, out_s, out_u;             // the CTA's, for the cluster's first
  int out_before, out_n;
  int n;                                 // listed (counted beyond kList)
  int n_best;
};

// Sum over the CTA of a small count; `flip` alternates between calls.
__device__ __forceinline__ int block_count(int c, Shared &sh, int &flip) {
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) sh.cnt[flip][threadIdx.x >> 5] = c;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += sh.cnt[flip][w];
  flip ^= 1;
  return t;
}

// Leaves in sh.best the k largest of the n keys in sh.list (all different, at
// most kList, n >= k), in no order; sh.n_best = k.  By bits from the top: the
// largest bound that at least k keys reach.
__device__ __forceinline__ void block_select(Shared &sh, int n, int k, int &flip) {
  constexpr int P = kList / kThreads;
  unsigned long long key[P];
  uint32_t hi = 0u, lo = ~0u;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = threadIdx.x + i * kThreads;
    key[i] = at < n ? sh.list[at] : 0ull;
    if (at < n) {
      hi = max(hi, static_cast<uint32_t>(key[i] >> 32));
      lo = min(lo, static_cast<uint32_t>(key[i] >> 32));
    }
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (threadIdx.x == 0) sh.n_best = 0;
  if ((threadIdx.x & 31) == 0) {
    sh.cnt[flip][threadIdx.x >> 5] = static_cast<int>(hi);
    sh.low[threadIdx.x >> 5] = lo;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    hi = max(hi, static_cast<uint32_t>(sh.cnt[flip][w]));
    lo = min(lo, sh.low[w]);
  }
  flip ^= 1;
  // bits above the first that differs between the smallest and largest are the bound's too
  int bit = hi == lo ? 31 : 63 - __clz(hi ^ lo);
  unsigned long long bound = (static_cast<unsigned long long>(hi) << 32) & ~((2ull << bit) - 1ull);
  int got = n;
  while (bit >= 0 && got != k) {
    const unsigned long long t = bound | (1ull << bit);
    int c = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) c += key[i] >= t;
    c = block_count(c, sh, flip);
    if (c >= k) {
      bound = t;
      got = c;
    }
    --bit;
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (key[i] >= bound && key[i] != 0ull) {
      const int at = atomicAdd(&sh.n_best, 1);
      if (at < kMaxTop) sh.best[at] = key[i];
    }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) score_kernel(const ScoreArgs a) {
  constexpr int W = Vec<T>::W, U = 4;
  constexpr int E = W * U;                // values of a thread and step
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t cr = cluster_rank(), cs = cluster_size();
  const int64_t row = blockIdx.x / cs;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  const int v = static_cast<int>(a.v), k = a.n_top;
  const float c = kLog2e / a.temperature;
  if (tid == 0) sh.n = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the logits are complete

  const int64_t tok = a.tokens ? a.tokens[row] : -1;
  const bool has = tok >= 0 && tok < v;
  // no value is above NaN: without a token nothing is counted
  const float xt = has ? to_float(x[tok]) : __int_as_float(0x7FFFFFFF);

  // this CTA's share: values [lo, hi) = head values (first CTA) + vectors [v0, v1) + the rest (last CTA)
  const RowCut cut = cut_row(x, v);
  const int v0 = static_cast<int>(static_cast<int64_t>(cut.vecs) * cr / cs);
  const int v1 = static_cast<int>(static_cast<int64_t>(cut.vecs) * (cr + 1) / cs);
  const uint32_t lo = cr == 0 ? 0 : cut.head + v0 * W;
  const uint32_t hi = cr == cs - 1 ? v : cut.head + v1 * W;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + cut.head);

  Stat st = {-INFINITY, 0.0f, 0.0f};
  float ref = 0.0f;                       // st.m, or 0 while that is -infinity
  int before = 0, flip = 0;
  // Too few vectors for a bound (at most 63, and 14 values beside them): every value is listed.
  const bool all = min(v1 - v0, kThreads) < k;
  float tau = __int_as_float(0x7FFFFFFF); // the bound; NaN: none yet

  auto add_max = [&](float cm) {
    if (cm > st.m) {
      const float d = (st.m - cm) * c, f = exp2_approx(d);
      st.u = st.s == 0.0f ? 0.0f : (st.u + st.s * fmaxf(d, -1e30f)) * f;
      st.s = st.m == -INFINITY ? st.s : st.s * f;   // -infinity seen alone left 0, a NaN stays
      st.m = ref = cm;
    }
  };
  auto add = [&](float xi) {
    const float d = (xi - ref) * c, e = exp2_approx(d);
    st.s += e;
    st.u = fmaf(e, fmaxf(d, -200.0f), st.u);        // 2^-200 is 0 here, and 0 times -infinity would be NaN
  };
  auto list = [&](float xi, int i) {
    if (*reinterpret_cast<volatile int *>(&sh.n) > kList) return;   // lost already: no queue at the counter
    const int at = atomicAdd(&sh.n, 1);
    if (at < kList) sh.list[at] = argmax_key(xi, static_cast<uint32_t>(i));
  };
  // the bound: largest key (its upper 16 bits) that at least k of the threads' maxima reach
  auto take_bound = [&]() {
    const uint32_t mine = v0 + tid < v1 ? float_order_key(st.m) : 0u;
    uint32_t b = 0u;
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t t = b | (1u << bit);
      if (__syncthreads_count(mine >= t) >= k) b = t;
    }
    tau = order_key_float(b < kKeyMinusInf ? kKeyMinusInf : b);
  };
  // values at the bound are listed too, unless it is -infinity: masked values are too many
  auto listed = [&](float xi) { return all || xi > tau || (xi == tau && tau != -INFINITY); };

  // head and rest: at most one value a thread of the first and last CTA
  int edge_i = -1;
  float edge = -INFINITY;
  {
    const int rest = v - cut.head - cut.vecs * W;
    if (cr == 0 && tid < cut.head) edge_i = tid;
    if (cr == cs - 1 && tid >= 32 && tid < 32 + rest) edge_i = v - rest + tid - 32;
    if (edge_i >= 0) {
      edge = to_float(x[edge_i]);
      add_max(edge);
      add(edge);
      before = edge > xt || (edge == xt && edge_i < tok);
    }
  }

  const int steps = (v1 - v0 + kThreads * U - 1) / (kThreads * U);
  uint4 nxt[U];
  auto fetch = [&](int s) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int at = v0 + (s * U + j) * kThreads + tid;
      if (at < v1) nxt[j] = __ldcs(xv + at);
    }
  };
  if (steps > 0) fetch(0);
  for (int s = 0; s < steps; ++s) {
    uint4 cur[U];
#pragma unroll
    for (int j = 0; j < U; ++j) cur[j] = nxt[j];
    if (s + 1 < steps) fetch(s + 1);
    const int at0 = v0 + s * U * kThreads + tid;
    auto each = [&](auto &&f) {           // over this step's values of the thread
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int at = at0 + j * kThreads;
        if (at < v1) {
          float o[W];
          unpack(cur[j], o, T{});
          const int i0 = cut.head + at * W;
#pragma unroll
          for (int i = 0; i < W; ++i) f(o[i], i0 + i);
        }
      }
    };
    float cm = -INFINITY;
    each([&](float xi, int) { cm = fmaxf(cm, xi); });
    add_max(cm);
    each([&](float xi, int) { add(xi); });
    if (cm >= xt) each([&](float xi, int i) { before += xi > xt || (xi == xt && i < tok); });
    if (k > 0) {
      if (!all && (s & (s - 1)) == 0) take_bound();   // after step 0, 1, 2, 4, 8, ..
      if (listed(cm))
        each([&](float xi, int i) {
          if (listed(xi)) list(xi, i);
        });
    }
  }
  if (k > 0 && edge_i >= 0 && listed(edge)) list(edge, edge_i);

  // the CTA's sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat b;
    b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    b.u = __shfl_xor_sync(0xffffffffu, st.u, o);
    st = stat_join(st, b, c);
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) {
    sh.m[warp] = st.m;
    sh.s[warp] = st.s;
    sh.u[warp] = st.u;
    sh.before[warp] = before;
  }
  __syncthreads();
  if (warp == 0) {
    st = lane < kWarps ? Stat{sh.m[lane], sh.s[lane], sh.u[lane]} : Stat{-INFINITY, 0.0f, 0.0f};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      Stat b;
      b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
      b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
      b.u = __shfl_xor_sync(0xffffffffu, st.u, o);
      st = stat_join(st, b, c);
    }
    before = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.before[lane] : 0);
    if (lane == 0) {
      sh.out_m = st.m;
      sh.out_s = st.s;
      sh.out_u = st.u;
      sh.out_before = before;
    }
  }

  // the CTA's alternatives: sh.list holds n values, the k first of its share among them
  int n = sh.n;
  if (k > 0 && !all && (n > kList || n < k)) {
    uint32_t bound = float_order_key(tau);
    auto key_at = [&](uint32_t i) { return float_order_key(to_float(x[i])); };
    auto count_from = [&](uint32_t t) {
      int m = 0;
      for (uint32_t i = lo + tid; i < hi; i += kThreads) m += key_at(i) >= t;
      return block_count(m, sh, flip);
    };
    if (n > kList) {
      if (count_from(bound + 1) >= k) {   // rising values: the k-th largest key itself, bit by bit
        uint32_t b = 0u;
        for (int bit = 31; bit >= 0; --bit)
          if (count_from(b | (1u << bit)) >= k) b |= 1u << bit;
        bound = b;
      }
      __syncthreads();
      if (tid == 0) sh.n = 0;
      __syncthreads();
      for (uint32_t i = lo + tid; i < hi; i += kThreads)   // fewer than k lie above the bound
        if (key_at(i) > bound) list(to_float(x[i]), i);
      __syncthreads();
      n = sh.n;
    }
    // then the bound's equals, by index
    for (uint32_t base = lo; base < hi && n < k; base += kThreads) {
      const bool eq = base + tid < hi && key_at(base + tid) == bound;
      const uint32_t m = __ballot_sync(0xffffffffu, eq);
      if (lane == 0) sh.cnt[flip][warp] = __popc(m);
      __syncthreads();
      int at = n + __popc(m & ((1u << lane) - 1u)), sum = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += sh.cnt[flip][w];
        sum += sh.cnt[flip][w];
      }
      if (eq && at < k) sh.list[at] = argmax_key(order_key_float(bound), base + tid);
      n = min(n + sum, k);
      flip ^= 1;
    }
    __syncthreads();
  }
  if (cs > 1) {
    if (n > kList / kMaxCluster) {        // what the first CTA has room for from each
      block_select(sh, n, k, flip);
      n = k;
      if (tid < k) sh.list[tid] = sh.best[tid];
    }
    if (tid == 0) sh.out_n = n;
    cluster_sync();
    if (cr == 0) {
      if (warp == 0) {
        const uint32_t r = lane < static_cast<int>(cs) ? lane : 0;
        st = {peer_loadf(peer_addr(&sh.out_m, r)), peer_loadf(peer_addr(&sh.out_s, r)),
              peer_loadf(peer_addr(&sh.out_u, r))};
        before = static_cast<int>(peer_loadu(peer_addr(&sh.out_before, r)));
        if (lane >= static_cast<int>(cs)) {
          st = {-INFINITY, 0.0f, 0.0f};
          before = 0;
        }
#pragma unroll
        for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
          Stat b;
          b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
          b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
          b.u = __shfl_xor_sync(0xffffffffu, st.u, o);
          st = stat_join(st, b, c);
        }
        before = __reduce_add_sync(0xffffffffu, before);
      }
      // one warp a peer's list, behind the lists before it
      int at = 0;
      for (uint32_t r = 0; r < cs; ++r) {
        const int nr = static_cast<int>(peer_loadu(peer_addr(&sh.out_n, r)));
        if (r > 0 && r == static_cast<uint32_t>(warp)) {
          const uint32_t from = peer_addr(sh.list, r);
          for (int i = lane; i < nr; i += 32) sh.list[at + i] = peer_load64(from + 8 * i);
        }
        at += nr;
      }
      n = at;
    }
    cluster_sync();                       // the peers' shared memory has been read
    if (cr != 0) return;
    if (tid == 0) {
      sh.out_m = st.m;
      sh.out_s = st.s;
      sh.out_u = st.u;
      sh.out_before = before;
    }
  }
  __syncthreads();
  const float m = sh.out_m == -INFINITY ? 0.0f : sh.out_m, total = sh.out_s;
  const bool empty = total == 0.0f;       // nothing above -infinity
  const float logs = logf(total);
  if (tid == 0) {
    if (a.lse) a.lse[row] = empty ? -INFINITY : m / a.temperature + logs;
    if (a.entropy) a.entropy[row] = empty ? 0.0f : logs - kLn2 * (sh.out_u / total);
    if (a.logprob) a.logprob[row] = !has ? 0.0f : empty ? -INFINITY : (xt - m) / a.temperature - logs;
    if (a.rank) a.rank[row] = has ? sh.out_before : -1;
  }
  if (k == 0) return;
  const int got = min(n, k);
  if (n > k) {
    block_select(sh, n, k, flip);
  } else {
    if (tid < got) sh.best[tid] = sh.list[tid];
    __syncthreads();
  }
  if (tid < k) {
    int at = tid;
    int32_t id = -1;
    float lp = -INFINITY;
    if (tid < got) {
      const unsigned long long key = sh.best[tid];
      at = 0;
      for (int i = 0; i < got; ++i) at += sh.best[i] > key;
      id = static_cast<int32_t>(argmax_key_index(key));
      if (!empty) lp = (order_key_float(static_cast<uint32_t>(key >> 32)) - m) / a.temperature - logs;
    }
    a.top_ids[row * k + at] = id;
    a.top_logprobs[row * k + at] = lp;
  }
}

template <typename T>
cudaError_t launch_score_t(const ScoreArgs &a) {
  static std::atomic<unsigned long long> configured{0};   // one bit per device; host threads may race here
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(score_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  int cs = 1;
  while (cs < kMaxCluster && a.n * 2 * cs <= 2 * a.num_sms && a.v / (2 * cs) >= 2048) cs *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n * cs));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start before the previous grid ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, score_kernel<T>, a);
}

}  // namespace

cudaError_t launch_score(const ScoreArgs &a) {
  if (a.dtype == 0) return launch_score_t<float>(a);
  if (a.dtype == 1) return launch_score_t<__half>(a);
  return launch_score_t<__nv_bfloat16>(a);
}

}  // namespace muse
