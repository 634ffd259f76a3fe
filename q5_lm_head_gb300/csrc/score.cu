// Scores of finished logits: the log probability and rank of a given token,
// the normaliser, the entropy and the top alternatives of each row.
//
// For a row x of V logits, c = log2(e) / temperature and m near max x:
//     a_i = (x_i - m) c,  S = sum_i 2^a_i,  U = sum_i 2^a_i a_i
//     lse = ln 2 (m c + log2 S),  logprob(t) = ln 2 (a_t - log2 S),  entropy = ln 2 (log2 S - U / S)
// Ranks and alternatives order by (x descending, index ascending), on x itself:
// a division could merge neighbouring values.
//
// Bound: HBM (each logit is read once) for many rows, latency for a few: 1,024 rows of
// 202,048 f32 take 159 us, 5.2 TB/s (77 % of the measured copy rate); the last
// of their 1.7 rounds of CTAs fills two SMs of three.  A cluster of 1, 2, 4, 8 or
// 16 CTAs takes a row (about as many as give each SM one), each a contiguous share
// of its 16-byte vectors; a thread holds a reference m with S and U, and the CTAs'
// results are pushed into the first one's shared memory.  No global workspace, so
// calls may overlap.
//
// Alternatives: a thread's running maximum stands for an element of its own, so
// the n_top-th largest of the maxima (of groups of two or four threads) is a
// value that at least n_top elements reach.  Elements from that bound up go to a
// list in shared memory; the bound is taken after the first step, whose values
// are still in registers, and again after 3, 7, 15 .. steps, so a row lists
// about n_top log2(steps) elements.  A bound of -infinity (a masked row) lists
// what is above it only.  A list that is short then, or that overflowed (equal
// or rising values), is made up by scans over the row: the values above the
// bound, then its first equals by index.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kList = 2048;                      // listed elements of a CTA
constexpr int kMaxCluster = 16;
constexpr int kShort = kList / kMaxCluster;      // elements that a CTA hands on, and that are ranked directly
static_assert(kShort >= kMaxTop, "a CTA's own alternatives");
constexpr float kLowest = -3.402823466e38f;
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;   // float_order_key(-infinity): below it only NaNs

// Sums S and U against the reference m, a value of the row; m = -infinity:
// nothing above -infinity seen (S and U are then 0, or NaN).
struct Stat {
  float m, s, u;
};

__device__ __forceinline__ Stat stat_move(Stat t, float m, float c) {
  if (m == -INFINITY) return {m, t.s, t.u};
  const float d = shift_exponent(t.m, m, c), f = exp2_approx(d);   // 2^-200 is 0 here
  return {m, t.s * f, (t.u + t.s * fmaxf(d, -200.0f)) * f};
}

// Sum over the warp's lanes, in a fixed order, against the largest of their values `most`.
__device__ __forceinline__ Stat stat_warp(Stat t, float most, float c) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, float_order_key(most));
  t = stat_move(t, order_key_float(top), c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t.s += __shfl_xor_sync(0xffffffffu, t.s, o);
    t.u += __shfl_xor_sync(0xffffffffu, t.u, o);
  }
  return t;
}

template <int kThreads>
struct Shared {
  static constexpr int kWarps = kThreads / 32;
  unsigned long long list[kList];
  unsigned long long got[kList];                 // first CTA: kShort from each of the cluster's
  unsigned long long best[kMaxTop];
  float m[kWarps], s[kWarps], u[kWarps];
  int before[kWarps];
  uint32_t high[kWarps], low[kWarps];
  uint32_t group[kThreads / 2], bound;
  int cnt[2][kWarps];
  int place[kShort];
  float from_m[kMaxCluster], from_s[kMaxCluster], from_u[kMaxCluster];   // first CTA: the cluster's
  int from_before[kMaxCluster], from_n[kMaxCluster];
  int n;                                         // listed (counted beyond kList)
  int kept;                                      // of trim
};

// Sum over the CTA of a small count; `flip` alternates between calls.
template <int kThreads>
__device__ __forceinline__ int block_count(int c, Shared<kThreads> &sh, int &flip) {
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) sh.cnt[flip][threadIdx.x >> 5] = c;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += sh.cnt[flip][w];
  flip ^= 1;
  return t;
}

// Cuts the n keys of list (all different, at most kList) to at most kShort with
// the k largest among them; returns how many.  By bits from the top: the
// largest bound that at least k keys reach, until few enough do.
template <int kThreads>
__device__ __forceinline__ int trim(unsigned long long *list, int n, int k, Shared<kThreads> &sh, int &flip) {
  if (n <= kShort) return n;
  constexpr int P = kList / kThreads;
  unsigned long long key[P];
  uint32_t hi = 0u, lo = ~0u;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = threadIdx.x + i * kThreads;
    key[i] = at < n ? list[at] : 0ull;
    if (at < n) {
      hi = max(hi, static_cast<uint32_t>(key[i] >> 32));
      lo = min(lo, static_cast<uint32_t>(key[i] >> 32));
    }
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if ((threadIdx.x & 31) == 0) {
    sh.high[threadIdx.x >> 5] = hi;
    sh.low[threadIdx.x >> 5] = lo;
  }
  if (threadIdx.x == 0) sh.kept = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    hi = max(hi, sh.high[w]);
    lo = min(lo, sh.low[w]);
  }
  // bits above the first that differs between the smallest and largest are the bound's too
  int bit = hi == lo ? 31 : 63 - __clz(hi ^ lo);
  unsigned long long bound = (static_cast<unsigned long long>(hi) << 32) & ~((2ull << bit) - 1ull);
  int got = n;
  for (; bit >= 0 && got > kShort; --bit) {
    const unsigned long long t = bound | (1ull << bit);
    int c = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) c += key[i] >= t;
    c = block_count(c, sh, flip);
    if (c >= k) {
      bound = t;
      got = c;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (key[i] >= bound && key[i] != 0ull) {
      const int at = atomicAdd(&sh.kept, 1);
      if (at < kShort) list[at] = key[i];
    }
  __syncthreads();
  return min(got, kShort);
}

// The k largest of the n <= kShort keys of list, in order, to sh.best: a key's
// place is how many are larger, counted by two or four threads.
template <int kThreads>
__device__ __forceinline__ void rank_top(const unsigned long long *list, int n, int k, Shared<kThreads> &sh) {
  const int i = threadIdx.x % kShort, part = threadIdx.x / kShort;
  constexpr int kParts = kThreads / kShort;
  if (threadIdx.x < kShort) sh.place[threadIdx.x] = 0;
  __syncthreads();
  const unsigned long long mine = i < n ? list[i] : 0ull;
  int larger = 0;
  for (int j = n * part / kParts; j < n * (part + 1) / kParts; ++j) larger += list[j] > mine;
  if (larger) atomicAdd(&sh.place[i], larger);
  __syncthreads();
  if (threadIdx.x < n && sh.place[threadIdx.x] < k) sh.best[sh.place[threadIdx.x]] = mine;
  __syncthreads();
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) score_kernel(const ScoreArgs a) {
  constexpr int W = Vec<T>::W, kWarps = kThreads / 32;
  constexpr int kVecs = 4;                // 16-byte vectors of a thread and step
  __shared__ Shared<kThreads> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t cr = cluster_rank(), cs = cluster_size();
  const int cs_log = 31 - __clz(cs);      // a power of two
  const int64_t row = blockIdx.x >> cs_log;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  const int v = static_cast<int>(a.v), k = a.n_top;
  const float c = a.exponent_scale;       // log2(e) / temperature
  if (cs > 1) cluster_arrive();           // waited for before the first store to a peer
  if (tid == 0) sh.n = 0;
  __syncthreads();

  // this CTA's share: values [lo, hi) = head values (first CTA) + vectors [v0, v1) + the rest (last CTA)
  const RowCut cut = cut_row(x, v);
  const int v0 = static_cast<int>((static_cast<int64_t>(cut.vecs) * cr) >> cs_log);
  const int v1 = static_cast<int>((static_cast<int64_t>(cut.vecs) * (cr + 1)) >> cs_log);
  const uint32_t lo = cr == 0 ? 0 : cut.head + v0 * W;
  const uint32_t hi = cr == cs - 1 ? v : cut.head + v1 * W;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + cut.head);
  const int steps = (v1 - v0 + kThreads * kVecs - 1) / (kThreads * kVecs);

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the logits are complete
  // full steps, in which every thread has kVecs vectors, and a last one with fewer
  const int full = (v1 - v0) / (kThreads * kVecs);
  uint4 nxt[kVecs];
  auto fetch = [&](int s) {
    const uint4 *p = xv + v0 + s * kVecs * kThreads + tid;
    if (s < full) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) nxt[j] = __ldcs(p + j * kThreads);
    } else {
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (v0 + (s * kVecs + j) * kThreads + tid < v1) nxt[j] = __ldcs(p + j * kThreads);
    }
  };
  if (steps > 0) fetch(0);
  const int64_t tok = a.tokens ? a.tokens[row] : -1;
  const bool has = tok >= 0 && tok < v;
  // no value reaches NaN: without a token nothing is counted
  const float xt = has ? to_float(x[tok]) : __int_as_float(0x7FFFFFFF);
  // the least value above xt: behind the token only those count
  const float xt_up = nextafterf(xt, INFINITY);

  // The sums' reference is the first maximum seen, and a later one only where it
  // lies 2^16 above: moving the sums onto every new maximum was most of a step's
  // instructions (some thread of a warp has one in three steps of four; with 2^8
  // 1,024 rows of 202,048 f32 take 3 % longer).  Each power of two
  // of that room costs the entropy of a nearly certain row 1e-7: log2 S and U / S
  // are that large, their difference small.
  Stat st = {-INFINITY, 0.0f, 0.0f};
  float ref = 0.0f, reach = -INFINITY;    // st.m, or 0 while that is -infinity; the largest value it serves
  float most = -INFINITY;                 // the thread's maximum
  const float room = 16.0f / c;
  unsigned long long s2 = 0ull, u2 = 0ull;   // two lanes of S and U
  int before = 0, flip = 0;
  // Groups of threads whose maxima give the bound: two or four threads, at
  // least n_top groups with a vector each; with fewer every value is listed
  // (at most 128 vectors and 14 values beside them).
  const int shift = k <= 32 ? 2 : 1;
  const bool all = min(v1 - v0, kThreads) < (k << shift);
  float bound = -INFINITY, lim = k > 0 && all ? -INFINITY : __int_as_float(0x7FFFFFFF);   // listed from lim up; NaN: nothing

  auto add_max = [&](float cm) {
    most = fmaxf(most, cm);
    if (cm > reach) {
      const float d = shift_exponent(st.m, cm, c), f = exp2_approx(d), low = fmaxf(d, -200.0f);   // as in stat_move
      u2 = mul2(fma2(s2, pack2(low, low), u2), pack2(f, f));
      s2 = mul2(s2, pack2(f, f));
      st.m = ref = cm;
      reach = cm + room;
    }
  };
  auto add = [&](float xi) {              // 2^-200 is 0 here, and 0 times -infinity would be NaN
    const float d = exponent(xi, ref, c), e = exp2_approx(d);
    s2 = add2(s2, pack2(e, 0.0f));
    u2 = fma2(pack2(e, 0.0f), pack2(fmaxf(d, -200.0f), 0.0f), u2);
  };
  auto list = [&](float xi, int i) {
    if (*reinterpret_cast<volatile int *>(&sh.n) > kList) return;   // lost already: no queue at the counter
    const int at = atomicAdd(&sh.n, 1);
    if (at < kList) sh.list[at] = argmax_key(xi + 0.0f, static_cast<uint32_t>(i));   // 0 and -0 are one value
  };
  // the largest key (its upper 16 bits) that at least k groups' maxima reach
  auto take_bound = [&]() {
    uint32_t mine = v0 + tid < v1 ? float_order_key(most) : 0u;
    mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
    if (shift == 2) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, 2));
    if ((tid & ((1 << shift) - 1)) == 0) sh.group[tid >> shift] = mine;
    __syncthreads();
    if (warp == 0) {                      // one warp: sixteen doing the same would cost issue slots
      constexpr int kKeys = kThreads / 64;   // of a lane, with groups of two threads
      uint32_t key[kKeys], top = 0u, low = ~0u;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        key[i] = i < kKeys / 2 || shift == 1 ? sh.group[lane + 32 * i] : 0u;
        top = max(top, key[i]);
        if (i < kKeys / 2 || shift == 1) low = min(low, key[i]);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      low = __reduce_min_sync(0xffffffffu, low);
      int bit = top == low ? 0 : 31 - __clz(top ^ low);
      uint32_t b = top == low ? top : top & ~((2u << bit) - 1u);
      for (; bit >= 16; --bit) {
        const uint32_t t = b | (1u << bit);
        int n = 0;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) n += key[i] >= t;
        if (__reduce_add_sync(0xffffffffu, n) >= k) b = t;
      }
      if (lane == 0) sh.bound = b;
    }
    __syncthreads();
    const uint32_t b = sh.bound;
    bound = order_key_float(b < kKeyMinusInf ? kKeyMinusInf : b);
    lim = fmaxf(bound, kLowest);
  };

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

  const unsigned long long c2 = pack2(c, c);
  // One step: kVecs vectors of the thread, or the first `mine` of them (kFull false).
  auto step = [&](const uint4 (&cur)[kVecs], int s, auto full_const) {
    constexpr bool kFull = decltype(full_const)::value;
    const int at0 = v0 + s * kVecs * kThreads + tid;
    const int mine = kFull ? kVecs : min(kVecs, (v1 - at0 + kThreads - 1) / kThreads);   // may be <= 0
    float top[kVecs], cm = -INFINITY;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      top[j] = -INFINITY;
      if (kFull || j < mine) {
        float o[W];
        unpack(cur[j], o, T{});
        top[j] = o[0];
#pragma unroll
        for (int i = 1; i < W; ++i) top[j] = fmaxf(top[j], o[i]);
      }
      cm = fmaxf(cm, top[j]);
    }
    add_max(cm);
    const float rc = -__fmul_rn(ref, c);
    if (kFull && plain_product(rc)) {
      const unsigned long long rc2 = pack2(rc, rc);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float o[W];
        unpack(cur[j], o, T{});
#pragma unroll
        for (int i = 0; i < W; i += 2) {
          const float2 d = unpack2(fma2(pack2(o[i], o[i + 1]), c2, rc2));
          const unsigned long long e = pack2(exp2_approx(d.x), exp2_approx(d.y));
          s2 = add2(s2, e);
          u2 = fma2(e, pack2(fmaxf(d.x, -200.0f), fmaxf(d.y, -200.0f)), u2);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float o[W];
        unpack(cur[j], o, T{});
        if (j < mine) {
#pragma unroll
          for (int i = 0; i < W; ++i) add(o[i]);
        }
      }
    }
    if (cm >= xt) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        if (top[j] >= xt && j < mine) {
          float o[W];
          unpack(cur[j], o, T{});
          const int i0 = cut.head + (at0 + j * kThreads) * W;
          if (tok < i0 || tok >= i0 + W) {
            const float from = i0 < tok ? xt : xt_up;
#pragma unroll
            for (int i = 0; i < W; ++i) before += o[i] >= from;
          } else {
#pragma unroll
            for (int i = 0; i < W; ++i) before += o[i] >= (i0 + i < tok ? xt : xt_up);
          }
        }
      }
    }
    if (k > 0) {
      // after step 0, 2, 6, 14, ..; not for the last one's sake alone
      if (!all && ((s + 2) & (s + 1)) == 0 && (s == 0 || s + 1 < steps)) take_bound();
      if (cm >= lim) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          if (top[j] >= lim && j < mine) {
            float o[W];
            unpack(cur[j], o, T{});
            const int i0 = cut.head + (at0 + j * kThreads) * W;
#pragma unroll
            for (int i = 0; i < W; ++i)
              if (o[i] >= lim) list(o[i], i0 + i);
          }
        }
      }
    }
  };
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    uint4 cur[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) cur[j] = nxt[j];
    if (s + 1 < steps) fetch(s + 1);
    if (s < full) step(cur, s, std::true_type{});
    else step(cur, s, std::false_type{});
  }
  if (edge_i >= 0 && edge >= lim) list(edge, edge_i);

  // the CTA's sums
  {
    const float2 s = unpack2(s2), u = unpack2(u2);
    st.s = s.x + s.y;
    st.u = u.x + u.y;
  }
  st = stat_warp(st, most, c);
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
    st = stat_warp(st, st.m, c);
    before = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.before[lane] : 0);
  }

  // the CTA's alternatives: sh.list holds n values, the k first of its share among them
  int n = sh.n;
  if (k > 0 && !all && (n > kList || n < k)) {
    uint32_t key = float_order_key(bound);
    auto key_at = [&](uint32_t i) { return float_order_key(to_float(x[i]) + 0.0f); };
    auto count_from = [&](uint32_t t) {
      int m = 0;
      for (uint32_t i = lo + tid; i < hi; i += kThreads) m += key_at(i) >= t;
      return block_count(m, sh, flip);
    };
    if (n > kList) {
      if (count_from(key + 1) >= k) {     // rising values: the k-th largest key itself, bit by bit
        uint32_t b = 0u;
        for (int bit = 31; bit >= 0; --bit)
          if (count_from(b | (1u << bit)) >= k) b |= 1u << bit;
        key = b;
      }
      __syncthreads();
      if (tid == 0) sh.n = 0;
      __syncthreads();
      for (uint32_t i = lo + tid; i < hi; i += kThreads)   // fewer than k lie above the key
        if (key_at(i) > key) list(to_float(x[i]), i);
      __syncthreads();
      n = min(sh.n, k);
    }
    // then the key's equals, by index
    for (uint32_t base = lo; base < hi && n < k; base += kThreads) {
      const bool eq = base + tid < hi && key_at(base + tid) == key;
      const uint32_t m = __ballot_sync(0xffffffffu, eq);
      if (lane == 0) sh.cnt[flip][warp] = __popc(m);
      __syncthreads();
      int at = n + __popc(m & ((1u << lane) - 1u)), sum = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += sh.cnt[flip][w];
        sum += sh.cnt[flip][w];
      }
      if (eq && at < k) sh.list[at] = argmax_key(order_key_float(key), base + tid);
      n = min(n + sum, k);
      flip ^= 1;
    }
    __syncthreads();
  }
  if (cs > 1) {
    n = trim(sh.list, n, k, sh, flip);
    cluster_wait();                       // every CTA of the cluster has started
    const uint32_t to = peer_addr(sh.got, 0) + cr * kShort * 8u;
    if (tid < n) peer_store64(to + 8 * tid, sh.list[tid]);
    if (tid == 0) {
      peer_store32(peer_addr(&sh.from_m[cr], 0), __float_as_uint(st.m));
      peer_store32(peer_addr(&sh.from_s[cr], 0), __float_as_uint(st.s));
      peer_store32(peer_addr(&sh.from_u[cr], 0), __float_as_uint(st.u));
      peer_store32(peer_addr(&sh.from_before[cr], 0), static_cast<uint32_t>(before));
      peer_store32(peer_addr(&sh.from_n[cr], 0), static_cast<uint32_t>(n));
    }
    cluster_sync();
    if (cr != 0) return;
    if (warp == 0) {
      const bool in = lane < static_cast<int>(cs);
      st = in ? Stat{sh.from_m[lane], sh.from_s[lane], sh.from_u[lane]} : Stat{-INFINITY, 0.0f, 0.0f};
      st = stat_warp(st, st.m, c);
      before = __reduce_add_sync(0xffffffffu, in ? sh.from_before[lane] : 0);
    }
    if (k > 0) {                          // close the lists up
      n = 0;
      for (int r = 0; r < static_cast<int>(cs); ++r) {
        const int theirs = sh.from_n[r];
        if (r % kWarps == warp)
          for (int i = lane; i < theirs; i += 32) sh.list[n + i] = sh.got[r * kShort + i];
        n += theirs;
      }
    }
  }
  if (tid == 0) {
    sh.m[0] = st.m;
    sh.s[0] = st.s;
    sh.u[0] = st.u;
  }
  __syncthreads();
  const float total = sh.s[0], m = sh.m[0] == -INFINITY ? 0.0f : sh.m[0];
  const bool empty = total == 0.0f;       // nothing above -infinity
  const float logs = log2f(total);
  // From here a few values a row, in 64 bits: in log2's units a lowest value would overflow.
  // Differences of logits first: of 3.4e38 in size they would swallow the sum's logarithm.
  const double temperature = a.temperature, log_sum = row_log_sum(m, c, logs);
  auto logprob = [&](float xi) {
    return empty ? -INFINITY : static_cast<float>((static_cast<double>(xi) - m) / temperature - log_sum);
  };
  if (tid == 0) {
    if (a.lse) a.lse[row] = empty ? -INFINITY : static_cast<float>(m / temperature + log_sum);
    const float entropy = static_cast<float>(kLn2) * (logs - sh.u[0] / total);
    if (a.entropy) a.entropy[row] = empty || entropy < 0.0f ? 0.0f : entropy;   // a NaN stays one
    if (a.logprob) a.logprob[row] = has ? logprob(xt) : 0.0f;
    if (a.rank) a.rank[row] = has ? before : -1;
  }
  if (k == 0) return;
  n = trim(sh.list, n, k, sh, flip);
  rank_top(sh.list, n, k, sh);
  if (tid < k) {
    int32_t id = -1;
    float lp = -INFINITY;
    if (tid < n) {
      const unsigned long long key = sh.best[tid];
      id = static_cast<int32_t>(argmax_key_index(key));
      lp = logprob(order_key_float(static_cast<uint32_t>(key >> 32)));
    }
    a.top_ids[row * k + tid] = id;
    a.top_logprobs[row * k + tid] = lp;
  }
}

template <typename T, int kThreads>
cudaError_t launch_score_t(const ScoreArgs &a, int cs) {
  static std::atomic<unsigned long long> configured{0};   // one bit per device; host threads may race here
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(score_kernel<T, kThreads>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
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
  return cudaLaunchKernelEx(&cfg, score_kernel<T, kThreads>, a);
}

// CTAs a row, and their threads (times in us for rows of 202,048 f32 and 8
// alternatives, by threads/CTAs a row; rows of 32,000 f32 and 50,257 bf16 order
// alike).  One CTA of 512 threads an SM (1 row: 512/16 11.5, 512/8 13.9, 512/1
// 32.7; 16 rows: 512/8 16.9, 512/16 19.8), or of 256 threads where a share is
// short (one row of 50,257 bf16: 256/8 9.8, 512/8 10.0, 512/16 11.2).  Where whole
// powers of two would leave a third of the SMs without one, smaller and more of
// them, two or three an SM (77 rows: 256/4 28.7, 512/2 30.4, 512/1 35.4).  Rows for
// more than one round of SMs: 153 rows 256/2 42.5, 512/1 47.0, 256/1 57.2; 304 rows
// 512/1 50.6, 256/2 56.2; beyond, four CTAs of 256 an SM, whose barriers fall into
// the others' loads (400 rows 256/1 73.8, 512/1 83.5).
template <typename T>
cudaError_t launch_score_rows(const ScoreArgs &a) {
  const int64_t n = a.n, sms = a.num_sms, bytes = a.v * static_cast<int64_t>(sizeof(T));
  constexpr int64_t kLeast = 8192, kShortShare = 16384;   // bytes of a CTA
  if (2 * n > 3 * sms) return n <= 2 * sms ? launch_score_t<T, 512>(a, 1) : launch_score_t<T, 256>(a, 1);
  if (n > sms) return launch_score_t<T, 256>(a, bytes >= 2 * kLeast ? 2 : 1);
  int cs = 1;
  while (cs < kMaxCluster && 2 * n * cs <= sms && bytes / (2 * cs) >= kLeast) cs *= 2;
  if (cs <= 2 && 3 * n * cs <= 2 * sms && bytes / (4 * cs) >= kLeast) return launch_score_t<T, 256>(a, 4 * cs);
  return bytes / cs < kShortShare ? launch_score_t<T, 256>(a, cs) : launch_score_t<T, 512>(a, cs);
}

}  // namespace

cudaError_t launch_score(const ScoreArgs &a) {
  if (a.dtype == 0) return launch_score_rows<float>(a);
  if (a.dtype == 1) return launch_score_rows<__half>(a);
  return launch_score_rows<__nv_bfloat16>(a);
}

}  // namespace muse
