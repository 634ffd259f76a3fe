// The next token of each row of logits, drawn from a given uniform number.
//
// For a row x of V logits, z = x / T, in the order (x descending, index ascending):
//     top-k   the first k
//     top-p   the entries of what top-k left before which less than p of its mass lies
//     min-p   those with (x - max x) / T >= log min_p
//     token   the lowest kept index i with  sum_{j <= i, kept} e^{z_j}  >  u * sum_{kept} e^{z_j}
// All three filters keep a beginning of that order, so what is kept is a threshold
// t with a number of its equals: every x > t, and the first `ties` x = t by index.
//
// A drawn token stands next to a border of the sums, and so does the last one that
// top-p keeps: sums in 32 bits would move one row in a few thousand to the
// neighbouring token.  Weights are therefore whole numbers, 2^38 for 2^E (E the
// largest logit's exponent in log2 units), and sums of them are exact in any order:
//     y = x log2(e) / T = E + e + i/512 + v/512,   |v| <= 1/2,  e <= 0
//     weight = 2^e 2^(i/512) (1 + p(v)),  2^(i/512) from a table in two f32 pieces,
// where y's fraction comes from one exact fma and p from a polynomial of degree
// two (2^-36 off at most).  The error of a weight is about 2^-35 of it, and 2^-39
// of 2^E; the same logit always has the same weight.  A row whose exponents pass
// 2^13 (a low temperature, or logits of 1e5) takes its weights in 64 bits.
//
// Bound: HBM for many rows, latency for a few.  A cluster of CTAs holds a row in its
// shared memory, each CTA a contiguous share, each warp a contiguous part of that, so
// that prefix sums over warps and CTAs follow the index.  The thresholds are found
// by histograms over the ordered bits of the logits (11, 11, 10 bits).  Nothing is
// kept in global memory, so calls may overlap.  A row that 16 CTAs cannot hold is
// read again for each pass.
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 16;
constexpr int kBins = 2048;
constexpr int kHeldTwo = 72 * 1024;      // bytes of a row in a CTA: two CTAs an SM
constexpr int kHeldOne = 184 * 1024;     // one CTA an SM

constexpr int kSteps = 512;              // table: 2^(i / 512)
constexpr int kFraction = 38;            // fractional bits of a weight
constexpr float kShift = 12582912.0f;    // 1.5 * 2^23: adding it rounds to a whole number
constexpr float kRound = 192.0f * 274877906944.0f;   // 1.5 * 2^7 * 2^38: adding it rounds to 2^-16 * 2^38
constexpr int kRoundBits = kFraction - 16;
constexpr float kOrders = 42.0f;         // a weight of 2^-42 is 0
// p(v) = 2^(v / 512) - 1: the cubic term, (ln 2 / 512)^3 / 6 v^3, goes into the linear one as its best
// linear fit on |v| <= 1/2, 3/16 v
constexpr double kP1 = 0.6931471805599453 / kSteps;
constexpr float kPoly1 = static_cast<float>(kP1 + kP1 * kP1 * kP1 / 32.0), kPoly2 = static_cast<float>(kP1 * kP1 / 2.0);

struct PowerTable {
  float2 at[kSteps];
};
constexpr double small_power(double y) {   // 2^y, |y| <= 1, by its series
  double term = 1.0, sum = 1.0;
  for (int i = 1; i < 24; ++i) {
    term *= y * 0.69314718055994530942 / i;
    sum += term;
  }
  return sum;
}
constexpr PowerTable make_powers() {
  PowerTable t = {};
  double coarse[16] = {}, fine[32] = {};
  for (int i = 0; i < 16; ++i) coarse[i] = small_power(i / 16.0);
  for (int i = 0; i < 32; ++i) fine[i] = small_power(i / 512.0);
  for (int i = 0; i < kSteps; ++i) {
    const double p = coarse[i / 32] * fine[i % 32];
    t.at[i].x = static_cast<float>(p);
    t.at[i].y = static_cast<float>(p - static_cast<double>(t.at[i].x));
  }
  return t;
}
__device__ const PowerTable kPowers = make_powers();

// What a row's weights need; of one row, the same in every CTA of its cluster.
struct Weigher {
  const float2 *table;
  float c1, c2;            // 512 log2(e) / T in two pieces
  float floor;             // logits are taken at least as large: weight 0
  uint32_t base;           // takes a whole number of 512ths to the bits of 2^(e + 38)
  bool wide;               // in 64 bits
  int drop;                // bits by which weights are shortened, so that 64 bits hold a row's sum
  float m;
  double c;                // log2(e) / T
};

__device__ __noinline__ unsigned long long wide_weight(float x, float m, double c) {
  const double d = (static_cast<double>(x) - m) * c;
  return d < -kOrders ? 0ull : static_cast<unsigned long long>(rint(exp2(d) * static_cast<double>(1ull << kFraction)));
}

// The weight's upper part, a multiple of 2^22, and the rest.
__device__ __forceinline__ void weight_parts(const Weigher &w, float x, uint32_t &high, int &low) {
  x = fmaxf(x, w.floor);
  const float q = fmaf(x, w.c1, kShift), whole = q - kShift;
  const float v = fmaf(x, w.c2, fmaf(x, w.c1, -whole));
  const float p = v * fmaf(v, kPoly2, kPoly1);
  const uint32_t bits = __float_as_uint(q);
  const float2 t = w.table[bits & (kSteps - 1)];
  const float s = __uint_as_float((bits & ~(kSteps - 1u)) * (1u << 14) + w.base);   // 2^(e + 38)
  const float a = t.x * s, up = a + kRound;
  high = __float_as_uint(up) - __float_as_uint(kRound);
  low = __float2int_rn(fmaf(fmaf(t.x, p, t.y), s, a - (up - kRound)));
}
template <bool kShort>                    // rows of at most 2^24 values
__device__ __forceinline__ unsigned long long weight(const Weigher &w, float x) {
  unsigned long long r;
  if (w.wide) {
    r = wide_weight(x, w.m, w.c);
  } else {
    uint32_t high;
    int low;
    weight_parts(w, x, high, low);
    r = (static_cast<unsigned long long>(high) << kRoundBits) + static_cast<long long>(low);
  }
  return kShort ? r : r >> w.drop;
}

// floor(f k), or the next whole number up, of 0 < f < 1.
__device__ __forceinline__ unsigned long long part_of(float f, unsigned long long k, bool up) {
  const uint32_t bits = __float_as_uint(f);
  const int s = 150 - static_cast<int>(bits >> 23);              // f = man 2^-s
  const unsigned long long man = (bits & 0x7FFFFFu) | 0x800000u;
  if (bits < 0x00800000u) return up;                             // below 2^-126
  const unsigned long long hi = __umul64hi(k, man), lo = k * man;
  unsigned long long r, rest;
  if (s < 64) {
    r = (hi << (64 - s)) | (lo >> s);
    rest = lo << (64 - s);
  } else {
    r = s == 64 ? hi : (s < 128 ? hi >> (s - 64) : 0ull);
    rest = lo | (s == 64 ? 0ull : (s < 128 ? hi << (128 - s) : hi));
  }
  return r + (up && rest != 0ull);
}

__device__ __forceinline__ float max_nan(float a, float b) {     // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Where the running count or mass of a histogram reaches a target.
struct Cross {
  unsigned long long mass;               // before the bin
  uint32_t count, bin;
};

struct Shared {
  float2 table[kSteps];
  uint32_t count[kBins], low[kBins], high[kBins];   // histogram: elements, their weights' sum in two words
  Weigher w;
  float row_max[kWarps];
  unsigned long long warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  Cross cross;
  // from the cluster's CTAs
  float from_max[kCluster];
  unsigned long long from_total[kCluster];
  unsigned long long slice_mass[kCluster];
  uint32_t slice_count[kCluster];
  unsigned long long from_mass[kCluster];
  uint32_t from_ties[kCluster];
};

__device__ __forceinline__ uint32_t peer_load32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Adds a weight to a bin: two 32-bit sums with the carry.
__device__ __forceinline__ void add_mass(Shared &sh, uint32_t bin, unsigned long long w) {
  const uint32_t lo = static_cast<uint32_t>(w);
  uint32_t hi = static_cast<uint32_t>(w >> 32);
  const uint32_t old = atomicAdd(&sh.low[bin], lo);
  hi += old + lo < old;
  if (hi) atomicAdd(&sh.high[bin], hi);
}

// The first bin at which the cluster's histograms reach `target` (elements, or
// mass when by_mass), in every CTA; false when they do not.  Each CTA adds up a slice of the bins.
__device__ __forceinline__ bool find_cross(Shared &sh, bool by_mass, unsigned long long target, Cross &out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cr = cluster_rank(), cs = cluster_size(), slice = kBins / cs;
  const int per = slice > kThreads ? slice / kThreads : 1;
  cluster_sync();                         // the histograms are complete
  constexpr int kMost = kBins / kThreads;
  unsigned long long mass[kMost], sum = 0ull;
  uint32_t count[kMost], number = 0u;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    mass[i] = 0ull;
    count[i] = 0u;
    if (i < per && tid * per < slice) {
      const int bin = cr * slice + tid * per + i;
      for (int r = 0; r < cs; ++r) {
        count[i] += peer_load32(peer_addr(&sh.count[bin], r));
        mass[i] += (static_cast<unsigned long long>(peer_load32(peer_addr(&sh.high[bin], r))) << 32) +
                   peer_load32(peer_addr(&sh.low[bin], r));
      }
    }
    sum += mass[i];
    number += count[i];
  }
  unsigned long long upto = sum;
  uint32_t upto_n = number;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long a = __shfl_up_sync(0xffffffffu, upto, o);
    const uint32_t b = __shfl_up_sync(0xffffffffu, upto_n, o);
    if (lane >= o) {
      upto += a;
      upto_n += b;
    }
  }
  if (lane == 31) {
    sh.warp_mass[warp] = upto;
    sh.warp_count[warp] = upto_n;
  }
  __syncthreads();
  unsigned long long total = 0ull, before = upto - sum;
  uint32_t total_n = 0u, before_n = upto_n - number;
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) {
      before += sh.warp_mass[i];
      before_n += sh.warp_count[i];
    }
    total += sh.warp_mass[i];
    total_n += sh.warp_count[i];
  }
  if (tid < cs) {
    peer_store64(peer_addr(&sh.slice_mass[cr], tid), total);
    peer_store32(peer_addr(&sh.slice_count[cr], tid), total_n);
  }
  cluster_sync();
  total = 0ull;
  total_n = 0u;
  for (int r = 0; r < cs; ++r) {
    if (r < cr) {
      before += sh.slice_mass[r];
      before_n += sh.slice_count[r];
    }
    total += sh.slice_mass[r];
    total_n += sh.slice_count[r];
  }
  if ((by_mass ? total : total_n) < target) return false;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (i < per && tid * per < slice) {
      const unsigned long long b = by_mass ? before : before_n, in = by_mass ? mass[i] : count[i];
      if (b < target && b + in >= target)
        for (int r = 0; r < cs; ++r) {
          peer_store64(peer_addr(&sh.cross.mass, r), before);
          peer_store32(peer_addr(&sh.cross.count, r), before_n);
          peer_store32(peer_addr(&sh.cross.bin, r), cr * slice + tid * per + i);
        }
    }
    before += mass[i];
    before_n += count[i];
  }
  cluster_sync();
  out = sh.cross;
  return true;
}

template <typename T, bool kHeld>
__global__ void __launch_bounds__(kThreads, kHeld ? 2 : 4) sample_kernel(const SampleArgs a) {
  constexpr int W = Vec<T>::W;
  extern __shared__ __align__(16) uint8_t held[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cr = cluster_rank(), cs = cluster_size(), cs_log = 31 - __clz(cs);
  const int64_t row = blockIdx.x >> cs_log;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  const int64_t v = a.v;
  cluster_arrive();                       // waited for before the first store to a peer

  // the row as 16-byte vectors from the boundary at or before its first value
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15) / static_cast<int>(sizeof(T));
  const T *x0 = x - off;
  const int64_t vecs = (off + v + W - 1) / W;
  const int64_t v0 = (vecs * cr) >> cs_log, v1 = (vecs * (cr + 1)) >> cs_log;
  // this warp's part of this CTA's share
  const int64_t w0 = v0 + (((v1 - v0) * warp) / kWarps), w1 = v0 + (((v1 - v0) * (warp + 1)) / kWarps);
  uint4 *vec_held = reinterpret_cast<uint4 *>(held);
  const auto whole = [&](int64_t i) { return i * W >= off && (i + 1) * W <= off + v; };
  const auto edge = [&](int64_t i) {      // a vector that the row only begins or ends in
    float o[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int64_t at = i * W + e - off;
      o[e] = at >= 0 && at < v ? to_float(x[at]) : -INFINITY;
    }
    return pack_vec(o, T{});
  };
  const auto load = [&](int64_t i, float (&o)[W]) {
    if constexpr (kHeld) {
      unpack(vec_held[i - v0], o, T{});
    } else {
      unpack(whole(i) ? __ldg(reinterpret_cast<const uint4 *>(x0) + i) : edge(i), o, T{});
    }
  };
  for (int i = tid; i < kSteps; i += kThreads) sh.table[i] = kPowers.at[i];

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the logits and settings are complete
  if constexpr (kHeld) {
    for (int64_t i = w0 + lane; i < w1; i += 32) {
      uint4 *to = vec_held + (i - v0);
      if (whole(i))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                     "l"(reinterpret_cast<const uint4 *>(x0) + i)
                     : "memory");
      else
        *to = edge(i);
    }
  }
  float temperature = a.temperatures ? a.temperatures[row] : a.temperature;
  int64_t top_k = a.top_ks ? a.top_ks[row] : a.top_k;
  const float top_p = a.top_ps ? a.top_ps[row] : a.top_p, min_p = a.min_ps ? a.min_ps[row] : a.min_p;
  const float u = a.uniforms[row];
  bool bad = top_p != top_p || min_p != min_p;
  if (temperature == 0.0f || top_p <= 0.0f) top_k = 1;   // the first
  if (temperature == 0.0f) temperature = 1.0f;
  bad |= !(temperature >= 0x1p-20f && temperature <= 0x1p20f);
  const bool by_k = top_k > 0 && top_k < v, by_p = top_p < 1.0f && top_p > 0.0f;
  if constexpr (kHeld) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
  }

  // the row's maximum; a NaN stays one
  float m = -INFINITY;
  for (int64_t i = w0 + lane; i < w1; i += 32) {
    float o[W];
    load(i, o);
#pragma unroll
    for (int e = 0; e < W; ++e) m = max_nan(m, o[e]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sh.row_max[warp] = m;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) m = max_nan(m, sh.row_max[i]);
  cluster_wait();                         // every CTA of the cluster has started
  if (tid < cs) peer_store32(peer_addr(&sh.from_max[cr], tid), __float_as_uint(m));
  cluster_sync();
  for (int i = 0; i < cs; ++i) m = max_nan(m, sh.from_max[i]);
  if (bad || !(fabsf(m) < INFINITY)) {    // settings or logits that are not numbers, an infinity, or nothing at all
    if (cr == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = !bad && m == -INFINITY ? -INFINITY : NAN;
    }
    return;
  }
  if (tid == 0) {
    const double c = 1.4426950408889634 / temperature;
    Weigher w;
    w.table = sh.table;
    w.c1 = static_cast<float>(c * kSteps);
    w.c2 = static_cast<float>(c * kSteps - w.c1);
    w.floor = __double2float_rd(m - kOrders / c);
    w.wide = !(fmaxf(fabsf(m), fabsf(w.floor)) * w.c1 < 4000000.0f);
    w.drop = v > (int64_t{1} << 24) ? 40 - __clzll(v - 1) : 0;   // bits of v - 1 beyond 24
    w.m = m;
    w.c = c;
    const uint32_t top = __float_as_uint(fmaf(m, w.c1, kShift)) & ~(kSteps - 1u);
    w.base = ((127u + kFraction) << 23) - top * (1u << 14);
    sh.w = w;
    sh.row_max[0] = min_p > 0.0f ? __double2float_ru(m + temperature * log(min_p < 1.0f ? static_cast<double>(min_p) : 1.0)) : -INFINITY;
  }
  __syncthreads();
  const Weigher w = sh.w;
  const float least = sh.row_max[0];      // of min-p

  // thresholds of top-k and top-p
  float t = least;                        // kept: x > t, and the first `ties` x = t
  unsigned long long ties = ~0ull;
  unsigned long long mass_k = 0ull;       // of what top-k left
  const auto select = [&](bool by_mass, unsigned long long target, bool want_mass) {
    unsigned long long mass = 0ull;
    uint32_t key = 0u;                    // of ~float_order_key, from the top
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const uint32_t mask = level == 2 ? 1023u : 2047u, fixed = level == 0 ? 0u : level == 1 ? ~0u << 21 : ~0u << 10;
      for (int i = tid; i < kBins; i += kThreads) sh.count[i] = sh.low[i] = sh.high[i] = 0u;
      __syncthreads();
      for (int64_t i = w0 + lane; i < w1; i += 32) {
        float o[W];
        load(i, o);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const uint32_t k = ~float_order_key(o[e]);
          if (o[e] >= w.floor && (k & fixed) == key) {
            if (!by_mass) atomicAdd(&sh.count[(k >> shift) & mask], 1u);
            if (want_mass) add_mass(sh, (k >> shift) & mask, weight<kHeld>(w, o[e]));
          }
        }
      }
      Cross at;
      if (!find_cross(sh, by_mass, target, at)) return false;   // only at the first level
      target -= by_mass ? at.mass : at.count;
      mass += at.mass;
      key |= at.bin << shift;
    }
    const float edge_x = order_key_float(~key);
    const unsigned long long of_one = weight<kHeld>(w, edge_x);
    const unsigned long long many = by_mass ? (target + of_one - 1) / of_one : target;
    mass_k = mass + many * of_one;
    if (edge_x > t || (edge_x == t && many < ties)) {
      t = edge_x;
      ties = many;
    }
    return true;
  };
  const auto total_mass = [&](float from) {   // of this warp's x >= from
    unsigned long long s = 0ull;
    for (int64_t i = w0 + lane; i < w1; i += 32) {
      float o[W];
      load(i, o);
#pragma unroll
      for (int e = 0; e < W; ++e)
        if (o[e] >= from) s += weight<kHeld>(w, o[e]);
    }
    return warp_sum(s);
  };
  if (by_p || by_k) {
    bool all = !by_k;
    if (by_k) all = !select(false, static_cast<unsigned long long>(top_k), by_p);
    if (by_p) {
      if (all) {                          // the mass of the whole row
        const unsigned long long s = total_mass(w.floor);
        if (lane == 0) sh.warp_mass[warp] = s;
        __syncthreads();
        unsigned long long sum = 0ull;
        for (int i = 0; i < kWarps; ++i) sum += sh.warp_mass[i];
        if (tid < cs) peer_store64(peer_addr(&sh.from_total[cr], tid), sum);
        cluster_sync();
        mass_k = 0ull;
        for (int i = 0; i < cs; ++i) mass_k += sh.from_total[i];
      }
      const unsigned long long need = part_of(top_p, mass_k, true);
      if (need > 0ull) select(true, need, true);
    }
  }

  // kept masses and ties of warps, CTAs
  unsigned long long mass = 0ull;
  uint32_t equal = 0u;
  for (int64_t i = w0 + lane; i < w1; i += 32) {
    float o[W];
    load(i, o);
#pragma unroll
    for (int e = 0; e < W; ++e) {
      if (o[e] > t && o[e] >= w.floor) mass += weight<kHeld>(w, o[e]);
      equal += o[e] == t;
    }
  }
  mass = warp_sum(mass);
  equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();                        // of total_mass
  if (lane == 0) {
    sh.warp_mass[warp] = mass;
    sh.warp_count[warp] = equal;
  }
  __syncthreads();
  unsigned long long sum = 0ull;
  uint32_t sum_n = 0u;
  for (int i = 0; i < kWarps; ++i) {
    sum += sh.warp_mass[i];
    sum_n += sh.warp_count[i];
  }
  if (tid < cs) {
    peer_store64(peer_addr(&sh.from_mass[cr], tid), sum);
    peer_store32(peer_addr(&sh.from_ties[cr], tid), sum_n);
  }
  cluster_sync();
  const unsigned long long of_tie = t >= w.floor ? weight<kHeld>(w, t) : 0ull;
  const auto kept_ties = [&](uint32_t n, unsigned long long &left) {
    const unsigned long long k = n < left ? n : left;
    left -= k;
    return k * of_tie;
  };
  unsigned long long total = 0ull, left = ties;
  for (int i = 0; i < cs; ++i) total += sh.from_mass[i] + kept_ties(sh.from_ties[i], left);
  const unsigned long long target = u >= 1.0f ? total - 1 : u > 0.0f ? part_of(u, total, false) : 0ull;

  // the CTA and the warp in which the sum passes the target
  unsigned long long upto = 0ull, add = 0ull;
  left = ties;
  int at = 0;
  for (; at < cr; ++at) upto += sh.from_mass[at] + kept_ties(sh.from_ties[at], left);
  {
    unsigned long long l = left;
    add = sh.from_mass[cr] + kept_ties(sh.from_ties[cr], l);
  }
  if (target < upto || target >= upto + add) return;
  for (at = 0; at < warp; ++at) upto += sh.warp_mass[at] + kept_ties(sh.warp_count[at], left);
  {
    unsigned long long l = left;
    add = sh.warp_mass[warp] + kept_ties(sh.warp_count[warp], l);
  }
  if (target < upto || target >= upto + add) return;
  for (int64_t i = w0; i < w1; i += 32) {
    float o[W];
    unsigned long long sum_above = 0ull;
    uint32_t n = 0u;
    if (i + lane < w1) {
      load(i + lane, o);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        if (o[e] > t && o[e] >= w.floor) sum_above += weight<kHeld>(w, o[e]);
        n += o[e] == t;
      }
    }
    uint32_t n_upto = n;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const uint32_t b = __shfl_up_sync(0xffffffffu, n_upto, s);
      if (lane >= s) n_upto += b;
    }
    unsigned long long mine_left = left > n_upto - n ? left - (n_upto - n) : 0ull;
    const unsigned long long left_here = mine_left;
    unsigned long long l = mine_left;
    const unsigned long long lane_sum = sum_above + kept_ties(n, l);
    unsigned long long s_upto = lane_sum;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const unsigned long long b = __shfl_up_sync(0xffffffffu, s_upto, s);
      if (lane >= s) s_upto += b;
    }
    unsigned long long here = upto + s_upto - lane_sum;
    if (target >= here && target < here + lane_sum) {
      unsigned long long tie = left_here;
      for (int e = 0; e < W; ++e) {
        unsigned long long k = 0ull;
        if (o[e] > t && o[e] >= w.floor) k = weight<kHeld>(w, o[e]);
        else if (o[e] == t && tie > 0ull) {
          --tie;
          k = of_tie;
        }
        if (target < here + k) {
          a.tokens[row] = static_cast<int32_t>((i + lane) * W + e - off);
          if (a.logprobs)
            a.logprobs[row] = static_cast<float>((static_cast<double>(o[e]) - m) / temperature -
                                                 log(static_cast<double>(total) / static_cast<double>(weight<kHeld>(w, m))));
          break;
        }
        here += k;
      }
    }
    upto += __shfl_sync(0xffffffffu, s_upto, 31);
    n_upto = __shfl_sync(0xffffffffu, n_upto, 31);
    left = left > n_upto ? left - n_upto : 0ull;
    if (upto > target) return;
  }
}

template <typename T, bool kHeld>
cudaError_t launch_sample_t(const SampleArgs &a, int cs, size_t shared) {
  static std::atomic<unsigned long long> configured{0};   // one bit per device; host threads may race here
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(sample_kernel<T, kHeld>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && kHeld)
      e = cudaFuncSetAttribute(sample_kernel<T, kHeld>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldOne);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n * cs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start before the previous grid ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (shared > kHeldTwo) {                // up to 16 SMs of one GPC at a time: not every device has them
    int fit = 0;
    e = cudaOccupancyMaxActiveClusters(&fit, sample_kernel<T, kHeld>, &cfg);
    if (e != cudaSuccess) return e;
    if (fit < 1) return launch_sample_t<T, false>(a, 8, 0);
  }
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, kHeld>, a);
}

template <typename T>
cudaError_t launch_sample_rows(const SampleArgs &a) {
  const int64_t vecs = a.v / Vec<T>::W + 2;
  auto held = [&](int64_t cs) { return (vecs + cs - 1) / cs * 16; };   // a share is at most this
  int cs = 1;
  while (cs < kCluster && held(cs) > kHeldTwo) cs *= 2;
  while (cs < kCluster && a.n * 2 * cs <= 2 * a.num_sms && a.v / (2 * cs) >= 2048) cs *= 2;
  if (held(cs) > kHeldOne || a.n * cs >= (int64_t{1} << 31)) return launch_sample_t<T, false>(a, a.n * 8 < (int64_t{1} << 31) ? 8 : 1, 0);
  return launch_sample_t<T, true>(a, cs, static_cast<size_t>(held(cs)));
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a) {
  if (a.dtype == 0) return launch_sample_rows<float>(a);
  if (a.dtype == 1) return launch_sample_rows<__half>(a);
  return launch_sample_rows<__nv_bfloat16>(a);
}

}  // namespace muse
