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
// Bound: for few rows latency (three cluster barriers with top-k or no filter, eight with top-p, and the passes'
// chains), for many the CUDA cores: one weight takes 20 instructions and a table look-up of six bank cycles, so all
// passes but that of an unfiltered row avoid them where they can.  A cluster of CTAs takes a row, each CTA a contiguous share, each warp a contiguous part of it,
// so that prefix sums over CTAs and warps follow the index.  A share is held in shared memory where that fits, else
// read again (from L2) by each pass.  The passes:
//   - the maximum, maxima of groups of threads, a sample.
//   - top-k up to 512 (few enough reach the bound up to about 300): the k-th largest of at least k maxima is a bound
//     that k values reach; what reaches it goes to
//     the first CTA, which does the rest with these few (1 row of 202,048 f32 with top-k 50 and top-p 11.0 us).
//   - no filter: the mass of the parts (16 rows 21 us).
//   - top-p: by the sample and the maxima the border lies in an octave or so.  Values from there up are summed as
//     weights, those in the octaves by a histogram of 1,024 bins, those below only about, by exponentials in 32 bits whose
//     error has a bound: of the row's mass they are 1 - p.  Then the bin in which the sum reaches p of the least and
//     of the most that the mass can be, and in one more pass its values, settled one by one.  Where the two differ (one
//     row in 13 of 202,048 bf16 values with 28,000 kept), the row's mass is summed as weights and the bin taken
//     again.  1,024 such rows 511 us; with weights for every value and pass 1,169, with histograms over the ordered bits 2,296.
//     A bin of more than 512 values is settled if they are all equal, as 16-bit logits far from 0 are (1,024 bf16 rows
//     around 8, top-p 0.9: 464 us with a deviation of 2.5, selected as below 3,373; with 0.5 803).
//   - the CTA in whose kept mass the number falls, its warp's part, its sixteenth, its value.
// What does not fit (top-k's border among equal logits by the hundred, a crowd of different ones in a bin, weights in
// 64 bits, top-k beyond some 300) is selected by histograms
// over the ordered bits of the logits, 10 bits at a time (1,024 bf16 rows with top-k 1,000 1,560 us, in 64 bits with
// top-p 2,620; 512 f32 rows with a deviation of 0.01 and top-p 3,260; one f32 row of these 38, 67, 108).
// Nothing is kept in global memory, so calls may overlap.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kOnly = 0, kFirst = 1, kSecond = 2;   // grids of a call
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCluster = 16;
constexpr int kBins = 1024;
constexpr int kFew = 512;                // values settled one by one
constexpr int kGroups = 512;             // maxima of groups
constexpr int kSample = 256;             // values of a warp that top-p's estimate takes
constexpr int kStaged = 2;               // 16-byte vectors of a lane and step, of rows in shared memory
constexpr int kRead = 4;                 // and of rows that are read again
constexpr int kQueue = 32 * 16 * kWarps; // bytes of the warps' queues, for each vector of a step
static_assert(kSample * 4 <= 32 * 16 * kStaged, "a warp's sample is in its queue");
constexpr int kHeldTwo = 72 * 1024;      // bytes of a row in a CTA and its queues: two CTAs an SM
constexpr int kHeldOne = 184 * 1024;     // one CTA an SM

constexpr int kSteps = 512;              // table: 2^(i / 512)
constexpr int kFraction = 38;            // fractional bits of a weight
constexpr float kShift = 12582912.0f;    // 1.5 * 2^23: adding it rounds to a whole number
constexpr float kRound = 192.0f * 274877906944.0f;   // 1.5 * 2^7 * 2^38: adding it rounds to 2^-16 * 2^38
constexpr int kRoundBits = kFraction - 16;
constexpr float kOrders = 42.0f;         // a weight of 2^-42 is 0
constexpr int kOctaves = 48;
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
  float c0, e;             // the same in 32 bits; E
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
// The same of two values at once.
__device__ __forceinline__ void weight_pair(const Weigher &w, float x0, float x1, uint32_t &high0, uint32_t &high1, int &low0, int &low1) {
  const unsigned long long x = pack2(fmaxf(x0, w.floor), fmaxf(x1, w.floor)), c1 = pack2(w.c1, w.c1), shift = pack2(kShift, kShift),
                           minus = pack2(-1.0f, -1.0f), round = pack2(kRound, kRound);
  const unsigned long long q = fma2(x, c1, shift), v = fma2(x, pack2(w.c2, w.c2), fma2(x, c1, fma2(q, minus, shift)));
  const unsigned long long p = mul2(v, fma2(v, pack2(kPoly2, kPoly2), pack2(kPoly1, kPoly1)));
  const float2 qf = unpack2(q);
  const uint32_t b0 = __float_as_uint(qf.x), b1 = __float_as_uint(qf.y);
  const float2 t0 = w.table[b0 & (kSteps - 1)], t1 = w.table[b1 & (kSteps - 1)];
  const unsigned long long s = pack2(__uint_as_float((b0 & ~(kSteps - 1u)) * (1u << 14) + w.base),
                                     __uint_as_float((b1 & ~(kSteps - 1u)) * (1u << 14) + w.base));
  const unsigned long long t = pack2(t0.x, t1.x), a = mul2(t, s), up = add2(a, round);
  const unsigned long long rest = add2(a, fma2(up, minus, round));
  const float2 low = unpack2(fma2(fma2(t, p, pack2(t0.y, t1.y)), s, rest)), upf = unpack2(up);
  high0 = __float_as_uint(upf.x) - __float_as_uint(kRound);
  high1 = __float_as_uint(upf.y) - __float_as_uint(kRound);
  low0 = __float2int_rn(low.x);
  low1 = __float2int_rn(low.y);
}
__device__ __forceinline__ unsigned long long whole_weight(uint32_t high, int low) {
  return (static_cast<unsigned long long>(high) << kRoundBits) + static_cast<long long>(low);
}
// A weight by itself.  Out of line: a kernel full of them waits for its own code.
__device__ __noinline__ unsigned long long weight(const Weigher &w, float x) {
  if (w.wide) return wide_weight(x, w.m, w.c) >> w.drop;
  uint32_t high;
  int low;
  weight_parts(w, x, high, low);
  return whole_weight(high, low) >> w.drop;
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

__device__ __forceinline__ uint32_t max_nan_word(uint32_t a, uint32_t b, float) {
  return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t max_nan_word(uint32_t a, uint32_t b, __half) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_word(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ uint4 vec_max_nan(const uint4 &a, const uint4 &b, T t) {
  return make_uint4(max_nan_word(a.x, b.x, t), max_nan_word(a.y, b.y, t), max_nan_word(a.z, b.z, t), max_nan_word(a.w, b.w, t));
}

// Where the running count or mass of a histogram reaches a target.
struct Cross {
  unsigned long long mass;               // before the bin
  uint32_t count, bin;
  uint32_t in, place;                    // values in the bin; of the CTAs before this one
};

// The least value of the logits' type from `v` up, in both halves of a word.
__device__ __forceinline__ float least_from(float v, float) { return v; }
__device__ __forceinline__ __half2 least_from(float v, __half) { return __half2half2(__float2half_ru(v)); }
__device__ __forceinline__ __nv_bfloat162 least_from(float v, __nv_bfloat16) { return __bfloat162bfloat162(__float2bfloat16_ru(v)); }
// Bits of a vector's values from there up: value e of vector j at bit 4 j + e, of 16-bit
// types at 4 j + e / 2 + 16 (e mod 2).  The vector keeps the others, -infinity for these.
__device__ __forceinline__ uint32_t values_from(uint4 &r, int j, float from) {
  uint32_t m = 0u;
  uint32_t *w = &r.x;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (__uint_as_float(w[i]) >= from) {
      m |= 1u << (4 * j + i);
      w[i] = 0xFF800000u;
    }
  return m;
}
template <typename T2>
__device__ __forceinline__ uint32_t values_from(uint4 &r, int j, T2 from) {
  constexpr uint32_t kNone = sizeof(T2) == 4 && std::is_same_v<T2, __half2> ? 0xFC00FC00u : 0xFF80FF80u;
  uint32_t m = 0u;
  uint32_t *w = &r.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t over = __hge2_mask(*reinterpret_cast<const T2 *>(&w[i]), from);
    m |= over & (0x00010001u << (4 * j + i));
    w[i] = (w[i] & ~over) | (kNone & over);
  }
  return m;
}
template <typename T>
__device__ __forceinline__ int vector_of(int bit) { return (bit & 15) >> 2; }
template <typename T>
__device__ __forceinline__ int value_of(int bit) { return sizeof(T) == 4 ? bit & 3 : 2 * (bit & 3) + (bit >> 4); }

struct __align__(16) Histogram {         // values, their weights' sum in two words
  uint32_t count[kBins], low[kBins], high[kBins];
};
struct Few {                             // values to settle one by one
  unsigned long long key[kFew], mass[kFew];
  float x[kFew];
};
struct Slice {                           // a CTA's bins of all CTAs' histograms
  unsigned long long mass[kBins];
  uint32_t number[kBins];
};
struct Edge {                            // top-p's last bin: all CTAs' values, and which warp this CTA's come from
  unsigned long long mass[kFew];
  float x[kFew];
  uint8_t warp[kFew];
};
struct Shared {
  float2 table[kSteps];
  union {                                // top-k does without a histogram
    Histogram h;
    Few few;
  };
  union {                                // a slice is of no use once the bin is known
    Slice slice;
    Edge edge;
    unsigned long long got[kBins];       // top-k's values, of all CTAs
  };
  uint16_t place[kBins];                 // of a slice's bin and a CTA: values of the CTAs before it, up to kFew
  uint32_t octave[2 * kOctaves];         // by the weight's power of two, in 256ths of it: sampled values; threads' maxima
  unsigned long long above[kWarps];      // mass of the warps' parts from a value up that is certainly kept
  float group[kGroups];                  // of the cluster
  Weigher w;
  double least_off, inv_t;               // T log(min_p), 1 / T
  float c_off;                           // w.c0 is off by, at most
  float bound, least;                    // of top-k, min-p
  int few_n;                             // listed
  uint32_t sampled;
  unsigned long long warp_mass[kWarps], warp_tail[kWarps];
  uint32_t warp_count[kWarps];
  float border;                          // settled: the threshold, how many of its equals, the mass up to there
  unsigned long long ties, reached;
  Cross cross;
  int cross_found;
  unsigned long long scan_mass[kWarps];
  uint32_t scan_count[kWarps];
  float lowest, guess, sure_guess;       // top-p's estimates
  unsigned long long above_all, need, need_most;
  unsigned long long total, target, upto, left, of_tie;   // of the draw
  int part;
  // from the cluster's CTAs
  unsigned long long from_total[kCluster], slice_mass[kCluster], from_mass[kCluster];
  uint32_t slice_count[kCluster], from_ties[kCluster], from_n[kCluster];
  unsigned long long from_tail[kCluster];
  uint32_t from_octave[kCluster][2 * kOctaves], from_sampled[kCluster];
};

__device__ __forceinline__ void peer_load128(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a) : "memory");
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the CTA; `out` [kWarps] is free again after the next barrier.
__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, unsigned long long *out) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) out[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0ull;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) v += out[i];
  return v;
}

// Adds a weight to a bin: two 32-bit sums with the carry.
__device__ __forceinline__ void add_mass(Shared &sh, uint32_t bin, unsigned long long w) {
  const uint32_t lo = static_cast<uint32_t>(w);
  uint32_t hi = static_cast<uint32_t>(w >> 32);
  const uint32_t old = atomicAdd(&sh.h.low[bin], lo);
  hi += old + lo < old;
  if (hi) atomicAdd(&sh.h.high[bin], hi);
}

// The first bin at which the cluster's histograms reach target() (values, or mass
// when by_mass), in every CTA; false when they do not.  To be called when all CTAs'
// histograms are complete.  Each CTA adds up a slice of the bins, a thread four bins of a CTA
// (single words from 16 CTAs took 8 us).  prepare() is for one warp that has none: target() may use what it wrote.
template <typename Prepare, typename Target>
__device__ __forceinline__ bool find_cross(Shared &sh, bool by_mass, const Prepare &prepare, const Target &target_of, Cross &out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cr = cluster_rank(), cs = cluster_size(), slice = kBins / cs;
  static_assert(kBins / 4 <= kThreads - 32, "a warp is left");
  if (tid < kBins / 4) {
    const int r = tid & (cs - 1), bin = tid / cs * 4, at = cr * slice + bin;
    uint32_t count[4], low[4], high[4];
    peer_load128(peer_addr(&sh.h.count[at], r), count);
    peer_load128(peer_addr(&sh.h.low[at], r), low);
    peer_load128(peer_addr(&sh.h.high[at], r), high);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t own = count[i];
      unsigned long long mass = (static_cast<unsigned long long>(high[i]) << 32) + low[i];
      for (int o = 1; o < cs; o <<= 1) {  // prefix sums over the CTAs
        const uint32_t n = __shfl_up_sync(0xffffffffu, count[i], o, cs);
        const unsigned long long s = __shfl_up_sync(0xffffffffu, mass, o, cs);
        if (r >= o) {
          count[i] += n;
          mass += s;
        }
      }
      sh.place[(bin + i) * cs + r] = static_cast<uint16_t>(min(count[i] - own, static_cast<uint32_t>(kFew)));
      if (r == cs - 1) {
        sh.slice.number[bin + i] = count[i];
        sh.slice.mass[bin + i] = mass;
      }
    }
  } else if (warp == kWarps - 1) {
    prepare();
  }
  __syncthreads();
  // a thread a bin of the slice, of a CTA by itself two
  const int each = slice > kThreads ? 2 : 1, bin = tid * each;
  static_assert(kBins <= 2 * kThreads, "two bins a thread");
  unsigned long long mass[2] = {0ull, 0ull}, upto = 0ull;
  uint32_t number[2] = {0u, 0u}, upto_n = 0u;
  if (warp * 32 * each < slice) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < each && bin + i < slice) {
        mass[i] = sh.slice.mass[bin + i];
        number[i] = sh.slice.number[bin + i];
      }
    upto = mass[0] + mass[1];
    upto_n = number[0] + number[1];
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long a = __shfl_up_sync(0xffffffffu, upto, o);
      const uint32_t b = __shfl_up_sync(0xffffffffu, upto_n, o);
      if (lane >= o) {
        upto += a;
        upto_n += b;
      }
    }
  }
  if (lane == 31) {
    sh.scan_mass[warp] = upto;
    sh.scan_count[warp] = upto_n;
  }
  __syncthreads();
  if (warp == 0) {
    const unsigned long long all = warp_sum(lane < kWarps ? sh.scan_mass[lane] : 0ull);
    const uint32_t all_n = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.scan_count[lane] : 0u);
    if (lane < cs) {
      peer_store64(peer_addr(&sh.slice_mass[cr], lane), all);
      peer_store32(peer_addr(&sh.slice_count[cr], lane), all_n);
    }
  }
  cluster_sync();
  if (warp * 32 * each < slice) {
    const unsigned long long target = target_of();
    const unsigned long long mine = lane < cs ? sh.slice_mass[lane] : 0ull;
    const uint32_t mine_n = lane < cs ? sh.slice_count[lane] : 0u;
    if (warp == 0) {
      const unsigned long long total = by_mass ? warp_sum(mine) : __reduce_add_sync(0xffffffffu, mine_n);
      if (lane == 0) sh.cross_found = total >= target;
    }
    // before the thread's bins: the slices of the CTAs before, the warps before, the lanes before
    static_assert(kWarps <= 16 && kCluster <= 16, "half a warp each");
    unsigned long long before = lane < cr ? mine : 0ull;
    uint32_t before_n = lane < cr ? mine_n : 0u;
    if (lane >= 16 && lane - 16 < warp) {
      before = sh.scan_mass[lane - 16];
      before_n = sh.scan_count[lane - 16];
    }
    before = warp_sum(before) + upto - mass[0] - mass[1];
    before_n = __reduce_add_sync(0xffffffffu, before_n) + upto_n - number[0] - number[1];
    int at = -1;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (at < 0) {
        const unsigned long long sum = by_mass ? before : before_n, one = by_mass ? mass[i] : number[i];
        if (sum < target && target <= sum + one) {
          at = bin + i;
        } else if (i == 0) {
          before += mass[0];
          before_n += number[0];
        }
      }
    const uint32_t here = __ballot_sync(0xffffffffu, at >= 0);
    if (here) {                           // a lane for each CTA
      const int from = __ffs(here) - 1;
      at = __shfl_sync(0xffffffffu, at, from);
      before = __shfl_sync(0xffffffffu, before, from);
      before_n = __shfl_sync(0xffffffffu, before_n, from);
      if (lane < cs) {
        peer_store64(peer_addr(&sh.cross.mass, lane), before);
        peer_store32(peer_addr(&sh.cross.count, lane), before_n);
        peer_store32(peer_addr(&sh.cross.bin, lane), cr * slice + at);
        peer_store32(peer_addr(&sh.cross.in, lane), sh.slice.number[at]);
        peer_store32(peer_addr(&sh.cross.place, lane), sh.place[at * cs + lane]);
      }
    }
  }
  cluster_sync();
  out = sh.cross;
  return sh.cross_found;
}

// Parts of a sum one behind another, a lane's each: `mass` and `count` equals of the threshold, of which `left` are
// still kept.  Returns the sum up to and with the lane's part; `add` is that part, `mine` what is left of the equals there.
__device__ __forceinline__ unsigned long long sum_parts(unsigned long long mass, uint32_t count, unsigned long long left,
                                                     unsigned long long of_tie, unsigned long long &add, unsigned long long &mine) {
  const int lane = threadIdx.x & 31;
  uint32_t upto = count;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += n;
  }
  upto -= count;
  mine = left > upto ? left - upto : 0ull;
  add = mass + (count < mine ? count : mine) * of_tie;
  unsigned long long sum = add;
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long n = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += n;
  }
  return sum;
}

// log(total / one) of whole numbers, total >= one: total against one 2^e 2^(i/512), with
// 2^(i/512) next below it from the table; what is left (below 2^-8) by its series.  The
// difference is taken in 64 bits, the rest of it has 32 bits of its own size.
__device__ __noinline__ double log_ratio(const float2 *table, unsigned long long total, unsigned long long one) {
  const float about = __log2f(static_cast<float>(total)) - __log2f(static_cast<float>(one));   // to 2^-16
  const int steps = max(static_cast<int>(about * kSteps), 0), e = steps / kSteps;
  const float2 t = table[steps % kSteps];
  const double scale = __longlong_as_double(static_cast<long long>(1023 + e) << 52);
  const double base = static_cast<double>(one) * (static_cast<double>(t.x) + t.y) * scale;
  const float f = static_cast<float>(static_cast<double>(total) - base) / static_cast<float>(base);
  return static_cast<double>(steps) * (0.6931471805599453 / kSteps) + static_cast<double>(f * fmaf(f, fmaf(f, 1.0f / 3.0f, -0.5f), 1.0f));
}

template <typename T, bool kHeld>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int W = Vec<T>::W;
  extern __shared__ __align__(16) uint8_t held[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cr = cluster_rank(), cs = cluster_size(), cs_log = 31 - __clz(cs);
  const int64_t row = blockIdx.x >> cs_log;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  const int64_t v = a.v;
  if (row >= a.n) {                       // behind the rows of a second grid: it ends no sooner than the first one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  cluster_arrive();                       // waited for before the first store to a peer

  // the row as 16-byte vectors from the boundary at or before its first value
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15) / static_cast<int>(sizeof(T));
  const T *x0 = x - off;
  const int64_t vecs = (off + v + W - 1) / W;
  const int v0 = static_cast<int>((vecs * cr) >> cs_log), v1 = static_cast<int>((vecs * (cr + 1)) >> cs_log);
  // a warp's part of this CTA's share
  const auto part_begin = [&](int i) { return v0 + static_cast<int>(static_cast<int64_t>(v1 - v0) * i / kWarps); };
  const int w0 = part_begin(warp), w1 = part_begin(warp + 1);
  uint4 *vec_held = reinterpret_cast<uint4 *>(held);
  constexpr int kVecs = kHeld ? kStaged : kRead;
  T *queue = reinterpret_cast<T *>(held + a.held_bytes) + warp * (kVecs * 32 * W);
  const int inner0 = off > 0, inner1 = static_cast<int>((off + v) / W);   // vectors that lie in the row entirely
  const auto whole = [&](int i) { return i >= inner0 && i < inner1; };
  const auto edge = [&](int i) {          // a vector that the row only begins or ends in
    float o[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int64_t at = static_cast<int64_t>(i) * W + e - off;
      o[e] = at >= 0 && at < v ? to_float(x[at]) : -INFINITY;
    }
    return pack_vec(o, T{});
  };
  const auto load_vec = [&](int i) {
    if constexpr (kHeld) return vec_held[i - v0];
    else return whole(i) ? reinterpret_cast<const uint4 *>(x0)[i] : edge(i);
  };
  const auto value_at = [&](int i, int e) {       // of a vector: -infinity beside the row
    if constexpr (kHeld) {
      return to_float(reinterpret_cast<const T *>(vec_held + (i - v0))[e]);
    } else {
      const uint32_t at = static_cast<uint32_t>(i) * W + e - off;
      return at < static_cast<uint32_t>(v) ? to_float(x[at]) : -INFINITY;
    }
  };
  for (int i = tid; i < kSteps; i += kThreads) sh.table[i] = kPowers.at[i];
  if (tid == 0) {
    sh.few_n = 0;
    sh.sampled = 0u;
  }
  if (tid < 2 * kOctaves) sh.octave[tid] = 0u;

  // The logits and settings are complete; so they are for a second grid, which starts when all CTAs of the first one have
  // come past here.
  if (a.grid != kSecond) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.grid == kFirst) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (kHeld) {
    for (int i = w0 + lane; i < w1; i += 32) {
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
  const bool by_k = top_k > 0 && top_k < v, by_p = top_p < 1.0f && top_p > 0.0f, by_m = min_p > 0.0f;
  // groups of top-k: as few of the CTA's threads in one as leave top_k groups in the cluster
  const bool few_k = by_k && top_k <= kFew && top_k <= static_cast<int64_t>(kThreads) * cs;
  int per_warp = 1;
  if (few_k)
    while (kWarps * cs * per_warp < top_k) per_warp *= 2;
  if (tid == 0) {                         // 64 bits take their time: beside the loads
    const double c = 1.4426950408889634 / temperature;
    sh.w.table = sh.table;
    sh.w.c1 = static_cast<float>(c * kSteps);
    sh.w.c2 = static_cast<float>(c * kSteps - sh.w.c1);
    sh.w.c = c;
    sh.w.c0 = static_cast<float>(c);
    sh.c_off = __double2float_ru(fabs(c - sh.w.c0) + 0x1p-50 * c);
    sh.w.drop = v > (int64_t{1} << 24) ? 40 - __clzll(v - 1) : 0;   // bits of v - 1 beyond 24
    sh.inv_t = c * 0.6931471805599453;
  }
  if (tid == 32) sh.least_off = by_m ? temperature * log(min_p < 1.0f ? static_cast<double>(min_p) : 1.0) : 0.0;
  if constexpr (kHeld) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();                         // a warp reads what it has fetched itself
  }

  // A step's vectors of a lane from vector i on; nothing beside the part.  Where all of a warp's lie inside row and part,
  // without a test of each (1,024 rows of 202,048 bf16 with top-p 581 us, tested one by one 640).
  const auto fetch = [&](int i, int end, uint4 (&r)[kVecs]) {
    const int first = i - lane, next = first + 32 * kVecs;
    if (!kHeld && first >= inner0 && next <= inner1 && next <= end) {
      const uint4 *p = reinterpret_cast<const uint4 *>(x0) + i;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) r[j] = p[32 * j];
      return;
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) r[j] = i + 32 * j < end ? load_vec(i + 32 * j) : vec_lowest(T{});
  };

  // The row's maximum, and those of its groups; a NaN stays one.  For top-p also a sample: some vectors' first values,
  // at most kSample of a warp, in its queue.
  const bool estimate = by_p && !by_k;
  const int apart = static_cast<int>((w1 - w0 + kSample - 1) / kSample);   // steps of which one is sampled
  uint32_t sampled = 0u;
  int samples = 0;
  float m = -INFINITY;
  {
    uint4 most = vec_lowest(T{});
    int step = 0;
    for (int i = w0 + lane; i - lane < w1; i += 32 * kVecs) {
      uint4 r[kVecs];
      fetch(i, w1, r);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) most = vec_max_nan(most, r[j], T{});
      if (estimate && --step < 0) {
        step = apart - 1;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
          if (samples < kSample / 32) {
            queue[samples++ * 32 + lane] = *reinterpret_cast<const T *>(&r[j]);
            sampled += i + 32 * j < w1;
          }
      }
    }
    float o[W];
    unpack(most, o, T{});
#pragma unroll
    for (int e = 0; e < W; ++e) m = max_nan(m, o[e]);
  }
  const float own = m;
  for (int o = 16; o >= per_warp; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  cluster_wait();                         // every CTA of the cluster has started
  for (int i = lane; i < cs * per_warp; i += 32)   // a lane's m is its group's, of lane i mod per_warp
    peer_store32(peer_addr(&sh.group[(cr * kWarps + warp) * per_warp + (i & (per_warp - 1))], i / per_warp), __float_as_uint(m));
  cluster_sync();
  const int groups = kWarps * cs * per_warp;
  m = -INFINITY;
  for (int i = lane; i < groups; i += 32) m = max_nan(m, sh.group[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (bad || !(fabsf(m) < INFINITY)) {    // settings or logits that are not numbers, an infinity, or nothing at all
    if (cr == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = !bad && m == -INFINITY ? -INFINITY : NAN;
    }
    return;
  }
  if (warp == 0) {
    float bound = -INFINITY;
    if (few_k) {                          // the largest value (its upper 16 bits) that top_k groups reach
      uint32_t key[kGroups / 32], high = 0u, low = ~0u;
#pragma unroll
      for (int i = 0; i < kGroups / 32; ++i) {
        key[i] = lane + 32 * i < groups ? float_order_key(sh.group[lane + 32 * i]) : 0u;
        high = max(high, key[i]);
        if (lane + 32 * i < groups) low = min(low, key[i]);
      }
      high = __reduce_max_sync(0xffffffffu, high);
      low = __reduce_min_sync(0xffffffffu, low);
      // bits above the first that differs are the bound's too; then two bits at a time
      int bit = high == low ? 0 : 31 - __clz(high ^ low);
      uint32_t b = high == low ? high : high & ~((2u << bit) - 1u);
      for (; bit >= 15; bit -= 2) {
        const uint32_t two = 1u << bit, one = two >> 1;
        uint32_t n = 0u;                  // of three bounds, 10 bits each
#pragma unroll
        for (int i = 0; i < kGroups / 32; ++i)
          n += (key[i] >= (b | one) ? 1u : 0u) + (key[i] >= (b | two) ? 1u << 10 : 0u) + (key[i] >= (b | two | one) ? 1u << 20 : 0u);
        n = __reduce_add_sync(0xffffffffu, n);
        if ((n >> 20) >= top_k) b |= two | one;
        else if (((n >> 10) & 1023u) >= top_k) b |= two;
        else if ((n & 1023u) >= top_k) b |= one;
      }
      bound = b < 0x00800000u ? -INFINITY : order_key_float(b);   // NaNs have no place here, -infinity is masked
    }
    if (lane == 0) {
      sh.w.floor = fmaxf(__fsub_rd(m, __fmul_ru(temperature, kOrders * 0.6931472f)), -3.402823466e38f);
      sh.w.wide = !(fmaxf(fabsf(m), fabsf(sh.w.floor)) * sh.w.c1 < 4000000.0f);
      sh.w.m = m;
      const uint32_t top = __float_as_uint(fmaf(m, sh.w.c1, kShift)) & ~(kSteps - 1u);
      sh.w.base = ((127u + kFraction) << 23) - top * (1u << 14);
      sh.w.e = (__uint_as_float(top) - kShift) * (1.0f / kSteps);
      sh.bound = fmaxf(bound, sh.w.floor);
      sh.least = by_m ? __double2float_ru(m + sh.least_off) : -INFINITY;
    }
  }
  __syncthreads();
  Weigher w = sh.w;
  w.table = sh.table;                     // known to be in shared memory here
  const float least = sh.least;

  const auto write = [&](float xi, uint32_t index, unsigned long long total) {
    a.tokens[row] = static_cast<int32_t>(index);
    if (a.logprobs)
      a.logprobs[row] = static_cast<float>((static_cast<double>(xi) - m) * sh.inv_t - log_ratio(sh.table, total, weight(sh.w, m)));
  };
  const auto drawn = [&](unsigned long long total) {
    return u >= 1.0f ? total - 1 : u > 0.0f ? part_of(u, total, false) : 0ull;
  };
  // the values of [from, to) of vectors [i0, i1), a few: each(value, index)
  const auto each_in = [&](int i0, int i1, float from, float to, auto &&each) {
    const auto least_in = least_from(from, T{}), least_over = least_from(to, T{});
    for (int i = i0 + lane; i - lane < i1; i += 32 * kVecs) {
      uint4 r[kVecs];
      fetch(i, i1, r);
      uint32_t some = 0u, over = 0u;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        uint4 low = r[j];
        some |= values_from(low, j, least_in);
      }
      if (__any_sync(0xffffffffu, some != 0u) == 0) continue;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) over |= values_from(r[j], j, least_over);
      for (some &= ~over; some != 0u; some &= some - 1) {
        const int bit = __ffs(some) - 1;
        const int at = i + 32 * vector_of<T>(bit);
        each(value_at(at, value_of<T>(bit)), static_cast<uint32_t>(at) * W + value_of<T>(bit) - off);
      }
    }
  };
  // The same of many, through the warp's queue, so that all lanes have two at a time: pair(value, value), the second
  // one -infinity where there is none, and done() after a step's.  look(vector)
  // at all of them, with -infinity for those of the range.
  const auto many_in = [&](int i0, int i1, float from, auto bounded, float to, auto &&look, auto &&pair, auto &&done) {
    const auto least_in = least_from(from, T{}), least_over = least_from(to, T{});
    for (int i = i0 + lane; i - lane < i1; i += 32 * kVecs) {
      uint4 r[kVecs];
      fetch(i, i1, r);
      uint32_t some = 0u;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        uint4 low = r[j];
        some |= values_from(low, j, least_in);
        look(low);
      }
      if constexpr (decltype(bounded)::value) {
        uint32_t over = 0u;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          uint4 low = r[j];
          over |= values_from(low, j, least_over);
        }
        some &= ~over;
      }
      const int many = __popc(some);
      int at = many;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int b = __shfl_up_sync(0xffffffffu, at, s);
        if (lane >= s) at += b;
      }
      const int all = __shfl_sync(0xffffffffu, at, 31);
      if (all > 0) {
        T *to_queue = queue + (at - many);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {   // bit by bit (a loop over those that are set is slower from a few on)
          const T *o = reinterpret_cast<const T *>(&r[j]);
#pragma unroll
          for (int e = 0; e < W; ++e)
            if (some & (1u << (sizeof(T) == 4 ? 4 * j + e : 4 * j + e / 2 + 16 * (e & 1)))) *to_queue++ = o[e];
        }
        __syncwarp();
        for (int k = lane; k < all; k += 64) pair(to_float(queue[k]), k + 32 < all ? to_float(queue[k + 32]) : -INFINITY);
        __syncwarp();
      }
      done();
    }
  };
  const auto nothing = [](const auto &...) {};

  // top-k: what reaches the bound, to the first CTA
  if (few_k) {
    const int room = kBins / cs;
    const uint32_t to = peer_addr(&sh.got[cr * room], 0);
    each_in(w0, w1, sh.bound, INFINITY, [&](float xi, uint32_t index) {
      const int at = atomicAdd(&sh.few_n, 1);
      if (at < room)
        peer_store64(to + 8 * at, (static_cast<unsigned long long>(__float_as_uint(xi)) << 32) | index);
    });
    __syncthreads();
    if (tid < cs) peer_store32(peer_addr(&sh.from_n[cr], tid), sh.few_n);
    cluster_sync();
    int n = 0;
    bool fits = true;
    for (int r = 0; r < cs; ++r) {
      fits &= sh.from_n[r] <= static_cast<uint32_t>(room);
      n += sh.from_n[r] <= static_cast<uint32_t>(room) ? static_cast<int>(sh.from_n[r]) : 0;
    }
    if (fits && n <= kFew) {
      if (cr != 0) return;
      if (tid < n) {
        int r = 0, at = tid;
        for (; at >= static_cast<int>(sh.from_n[r]); ++r) at -= sh.from_n[r];
        const unsigned long long entry = sh.got[r * room + at];
        const float xi = __uint_as_float(static_cast<uint32_t>(entry >> 32));
        sh.few.x[tid] = xi;
        sh.few.key[tid] = argmax_key(xi, static_cast<uint32_t>(entry));
        sh.few.mass[tid] = weight(sh.w, xi);
      }
      __syncthreads();
      // a value's place in the order and the mass before it, by some threads each
      int split = 1;
      while (split < 32 && 2 * split * n <= kThreads) split *= 2;
      const int i = tid / split, first = tid & (split - 1);
      unsigned long long key = 0ull, mine = 0ull, before = 0ull;
      float xi = 0.0f;
      int rank = 0;
      if (i < n) {
        key = sh.few.key[i];
        mine = sh.few.mass[i];
        xi = sh.few.x[i];
        for (int j = first; j < n; j += split)
          if (sh.few.key[j] > key) {
            ++rank;
            before += sh.few.mass[j];
          }
      }
      for (int o = split >> 1; o > 0; o >>= 1) {
        rank += __shfl_xor_sync(0xffffffffu, rank, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
      }
      bool keep = i < n && rank < top_k;
      const unsigned long long all = block_sum(keep && first == 0 ? mine : 0ull, sh.warp_mass);
      keep = keep && xi >= least && (!by_p || before < part_of(top_p, all, true));
      if (!keep) mine = 0ull;
      if (i < n && first == 0) sh.few.mass[i] = mine;
      const unsigned long long total = block_sum(first == 0 ? mine : 0ull, sh.from_total);
      static_assert(kCluster >= kWarps, "from_total serves as the CTA's sums");
      const unsigned long long target = drawn(total);
      before = 0ull;                      // by index: the key's lower half falls with it
      if (mine > 0ull)
        for (int j = first; j < n; j += split)
          if (static_cast<uint32_t>(sh.few.key[j]) > static_cast<uint32_t>(key)) before += sh.few.mass[j];
      for (int o = split >> 1; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      if (first == 0 && mine > 0ull && before <= target && target < before + mine) write(xi, argmax_key_index(key), total);
      return;
    }
  }

  // thresholds of top-k and top-p
  float t = least;                        // kept: x > t, and the first `ties` x = t
  unsigned long long ties = ~0ull;
  unsigned long long mass_k = 0ull;       // of what top-k left
  const auto lower = [&](float edge_x, unsigned long long many) {
    if (edge_x > t || (edge_x == t && many < ties)) {
      t = edge_x;
      ties = many;
    }
  };
  const auto clear = [&]() {
    for (int i = tid; i < kBins; i += kThreads) sh.h.count[i] = sh.h.low[i] = sh.h.high[i] = 0u;
    __syncthreads();
  };
  // by the ordered bits, 10 at a time
  const auto select = [&](bool by_mass, unsigned long long target, bool want_mass) {
    unsigned long long mass = 0ull;
    uint32_t key = 0u;                    // of ~float_order_key, from the top
#pragma unroll 1
    for (int level = 0; level < 4; ++level) {
      const int shift = level < 3 ? 22 - 10 * level : 0;
      const uint32_t mask = level < 3 ? 1023u : 3u, fixed = level == 0 ? 0u : ~0u << (32 - 10 * level);
      __syncthreads();
      clear();
      for (int i = w0 + lane; i < w1; i += 32) {
#pragma unroll 1
        for (int e = 0; e < W; ++e) {
          const float xi = value_at(i, e);
          const uint32_t k = ~float_order_key(xi);
          if (xi >= w.floor && (k & fixed) == key) {
            atomicAdd(&sh.h.count[(k >> shift) & mask], 1u);
            if (want_mass) add_mass(sh, (k >> shift) & mask, weight(sh.w, xi));
          }
        }
      }
      cluster_sync();
      Cross at;
      if (!find_cross(sh, by_mass, [] {}, [&] { return target; }, at)) return false;   // only at the first level
      target -= by_mass ? at.mass : at.count;
      mass += at.mass;
      key |= at.bin << shift;
    }
    const float edge_x = order_key_float(~key);
    const unsigned long long of_one = weight(sh.w, edge_x);
    const unsigned long long many = by_mass ? (target + of_one - 1) / of_one : target;
    mass_k = mass + many * of_one;
    lower(edge_x, many);
    return true;
  };
  // the mass of this warp's part
  const auto part_mass = [&]() {
    unsigned long long s = 0ull;
    if (w.wide || w.drop > 0) {
      for (int i = w0 + lane; i < w1; i += 32) {
#pragma unroll 1
        for (int e = 0; e < W; ++e) s += weight(sh.w, value_at(i, e));
      }
    } else {
      uint32_t highs = 0u;                // parts of at most 2^17 each
      long long lows = 0ll;
      int steps = 0;
      for (int i = w0 + lane; i - lane < w1; i += 32 * kVecs) {
        uint4 r[kVecs];
        fetch(i, w1, r);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          float o[W];
          unpack(r[j], o, T{});
#pragma unroll
          for (int e = 0; e < W; e += 4) {
            uint32_t high[4];
            int low[4];                   // below 2^29 each
            weight_pair(w, o[e], o[e + 1], high[0], high[1], low[0], low[1]);
            weight_pair(w, o[e + 2], o[e + 3], high[2], high[3], low[2], low[3]);
            highs += high[0] + high[1] + high[2] + high[3];
            lows += low[0] + low[1] + low[2] + low[3];
          }
        }
        if (++steps == 256) {             // 2^13 values
          s += static_cast<unsigned long long>(highs) << kRoundBits;
          highs = 0u;
          steps = 0;
        }
      }
      s += (static_cast<unsigned long long>(highs) << kRoundBits) + static_cast<unsigned long long>(lows);
    }
    return warp_sum(s);
  };
  // a CTA's sums, of its warps' in warp_mass and warp_count, to all CTAs
  const auto hand_round = [&]() {
    __syncthreads();
    if (warp == 0) {
      const unsigned long long sum = warp_sum(lane < kWarps ? sh.warp_mass[lane] : 0ull);
      const uint32_t n = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_count[lane] : 0u);
      if (lane < cs) {
        peer_store64(peer_addr(&sh.from_mass[cr], lane), sum);
        peer_store32(peer_addr(&sh.from_ties[cr], lane), n);
      }
    }
    cluster_sync();
  };
  // the mass of the parts, of the CTAs
  const auto row_mass = [&]() {
    const unsigned long long s = part_mass();
    __syncthreads();
    if (lane == 0) {
      sh.warp_mass[warp] = s;
      sh.warp_count[warp] = 0u;
    }
    hand_round();
  };
  const auto whole_mass = [&]() {
    row_mass();
    return warp_sum(lane < cs ? sh.from_mass[lane] : 0ull);
  };
  // the mass of the values above t of vectors [i0, i1), and how many equal it
  const auto part_kept = [&](int i0, int i1, uint32_t &equal) {
    unsigned long long s = 0ull;
    uint32_t n = 0u;
    many_in(
        i0, i1, fmaxf(t, w.floor), std::false_type{}, 0.0f, nothing,
        [&](float xi, float xj) {
          if (w.wide || w.drop > 0) {
            s += xi == t ? 0ull : weight(sh.w, xi);
            s += xj == t || xj == -INFINITY ? 0ull : weight(sh.w, xj);
          } else {
            uint32_t high[2];
            int low[2];
            weight_pair(w, xi == t ? -INFINITY : xi, xj == t ? -INFINITY : xj, high[0], high[1], low[0], low[1]);
            s += whole_weight(high[0] + high[1], low[0] + low[1]);
          }
          n += (xi == t) + (xj == t && xj > -INFINITY);
        },
        nothing);
    equal = __reduce_add_sync(0xffffffffu, n);
    return warp_sum(s);
  };

  const bool plain = !by_k && !by_p && !by_m;
  bool whole_row = !by_k;
  if (by_k) whole_row = !select(false, static_cast<unsigned long long>(top_k), by_p);
  if (plain) row_mass();
  bool kept_known = false;                // the warps' kept mass and ties are in sh.above and sh.warp_count
  if (by_p && whole_row && !w.wide && w.drop == 0) {
    // Where the row's mass lies, about: by octave from the sample and, as that has few of the largest values, from the
    // threads' maxima.
    const unsigned long long c2 = pack2(w.c0, w.c0), e2 = pack2(-w.e, -w.e);
    const auto into = [&](float xi, uint32_t *octave) {
      const uint32_t bits = __float_as_uint(exp2_approx(fmaf(xi, w.c0, -w.e)));
      const int o = max(127 - static_cast<int>(bits >> 23), 0);
      if (o < kOctaves) atomicAdd(octave + o, 256u + ((bits >> 15) & 255u));
    };
    into(own, sh.octave + kOctaves);
    for (int i = 0; i < samples; ++i) into(to_float(queue[i * 32 + lane]), sh.octave);
    sampled = __reduce_add_sync(0xffffffffu, sampled);
    if (lane == 0) atomicAdd(&sh.sampled, sampled);
    __syncthreads();
    for (int i = tid; i < cs * 2 * kOctaves; i += kThreads)
      peer_store32(peer_addr(&sh.from_octave[cr][i % (2 * kOctaves)], i / (2 * kOctaves)), sh.octave[i % (2 * kOctaves)]);
    if (tid < cs) peer_store32(peer_addr(&sh.from_sampled[cr], tid), sh.sampled);
    clear();
    cluster_sync();
    if (warp == 0) {
      float number = 0.0f, mine[2] = {0.0f, 0.0f}, largest = 0.0f;   // of the lane's two octaves
      bool known[2] = {false, false};
      for (int r = 0; r < cs; ++r) number += static_cast<float>(sh.from_sampled[r]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < kOctaves) {
          float some = 0.0f, high = 0.0f;
          for (int r = 0; r < cs; ++r) {
            some += static_cast<float>(sh.from_octave[r][lane + 32 * h]);
            high += static_cast<float>(sh.from_octave[r][kOctaves + lane + 32 * h]);
          }
          const float unit = exp2f(-8.0f - static_cast<float>(lane + 32 * h));
          // one of the largest in the sample would stand for many that are not there: 16 at least
          mine[h] = fmaxf(some >= 16.0f * 384.0f ? some * (static_cast<float>(v) / fmaxf(number, 1.0f)) : 0.0f, high) * unit;
          largest += high * unit;
          known[h] = some >= 128.0f * 384.0f;
        }
      float about = mine[0] + mine[1];
      for (int o = 16; o > 0; o >>= 1) {
        about += __shfl_xor_sync(0xffffffffu, about, o);
        largest += __shfl_xor_sync(0xffffffffu, largest, o);
      }
      // Below this a value cannot be the border: all such values together weigh less than 1 - p of the maxima alone.
      const float share = (1.0f - top_p) * largest / static_cast<float>(v);
      const float low = fmaxf(fmaxf(w.floor, least), fmaf(__log2f(share * 0.98f) + w.e, 1.0f / w.c0, -1e-4f * temperature - 1e-5f * fabsf(m)));
      // By the octaves, the border lies above where seven tenths of 1 - p lie below, and below where that is fourteen; a
      // border that is not there is not found there.
      float guess = low, sure_guess = INFINITY;
      {
        const float enough = (1.0f - top_p) * about;
        float below = 0.0f, upto[2];
        int low_cut = kOctaves, high_cut = -1;
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          float s = mine[h];
          for (int o = 1; o < 32; o <<= 1) {
            const float t = __shfl_down_sync(0xffffffffu, s, o);
            if (lane + o < 32) s += t;
          }
          // an octave and all below it
          const uint32_t little = __ballot_sync(0xffffffffu, s + below < 0.7f * enough), much = __ballot_sync(0xffffffffu, s + below > 1.4f * enough);
          if (little) low_cut = 32 * h + __ffs(little) - 1;
          if (much && high_cut < 0) high_cut = 32 * h + 31 - __clz(much);
          upto[h] = s + below;
          below += __shfl_sync(0xffffffffu, s, 0);
        }
        // where in octave o a mass lies below, about, as a part of it; `other` where the sample has few values of it
        const auto part = [&](int o, float mass, float other) {
          const float all = __shfl_sync(0xffffffffu, upto[o >> 5], o & 31), one = __shfl_sync(0xffffffffu, mine[o >> 5], o & 31);
          return __shfl_sync(0xffffffffu, known[o >> 5], o & 31) ? (mass - (all - one)) / one : other;
        };
        // with a quarter of the lower part less and a quarter of an octave more, as the mass need not be even in an octave
        if (low_cut < kOctaves) {
          const float in = low_cut > 0 ? fminf(fmaxf(0.75f * part(low_cut - 1, 0.7f * enough, 0.0f), 0.0f), 1.0f) : 0.0f;
          guess = fmaxf(low, (w.e - static_cast<float>(low_cut - 1) + in) / w.c0);
        }
        if (high_cut > 0) sure_guess = (w.e - static_cast<float>(high_cut) + fminf(fmaxf(0.25f + part(high_cut, 1.4f * enough, 1.0f), 0.0f), 1.0f)) / w.c0;
        if (!(sure_guess > guess)) sure_guess = INFINITY;
      }
      if (lane == 0) {
        sh.lowest = low;
        sh.guess = guess;
        sh.sure_guess = sure_guess;
      }
    }
    __syncthreads();
    const float lowest = sh.lowest, guess = sh.guess, sure_guess = sh.sure_guess;
    // What the mass below may be off by, of itself: an exponent's rounding (half the last place of numbers up to 32; below
    // 2^-32 of 2^E a weight has 64 units, and v units are added anyway), that of log2(e) / T, as it is, 2 ulp of an exponential, eight
    // additions, and the weights' own 2^-32.
    const float off_by = 0.6931472f * (0x1p-20f + fmaxf(fabsf(m), fabsf(m - 33.0f / w.c0)) * sh.c_off) + 0x1p-22f + 0x1.1p-21f + 0x1p-32f;
    bool settled = false, guessed = guess > lowest || sure_guess < INFINITY, found = false;
#pragma unroll 1
    for (int attempt = 0; attempt < 2 && !found; ++attempt) {
      const float from = guessed ? guess : lowest, top = guessed ? sure_guess : INFINITY, base = fminf(top, m);
      const float reach = base - from, scale = reach > 0.0f ? fminf((kBins - 0.5f) / reach, 1e30f) : 0.0f;
      const auto bin_of = [&](float xi) { return min(static_cast<int>((base - xi) * scale), kBins - 1); };
      if (attempt > 0) {
        cluster_sync();                   // all have read what came before
        clear();
      }
      if (tid == 0) sh.few_n = 0;
      // mass from `top` up, and from `from` up; what lies below, about
      unsigned long long above = 0ull, upper = 0ull, tail = 0ull, sum = 0ull;
      const auto binned = [&](float xi, uint32_t high, int low) {
        const unsigned long long one = whole_weight(high, low);
        above -= one;                     // of all, what goes into the histogram
        const int bin = bin_of(xi);
        atomicAdd(&sh.h.count[bin], 1u);
        add_mass(sh, bin, one);
      };
      many_in(
          w0, w1, from, std::false_type{}, 0.0f,
          [&](const uint4 &r) {
            float o[W];
            unpack(r, o, T{});
            unsigned long long of_vec = 0ull;   // at most three additions, four to the step's sum, one of its halves
#pragma unroll
            for (int e = 0; e < W; e += 2) {
              const float2 y = unpack2(fma2(pack2(o[e], o[e + 1]), c2, e2));
              const unsigned long long two = pack2(exp2_approx(y.x), exp2_approx(y.y));
              of_vec = e == 0 ? two : add2(of_vec, two);
            }
            sum = add2(sum, of_vec);
          },
          [&](float xi, float xj) {
            uint32_t high[2];
            int low[2];
            weight_pair(w, xi, xj, high[0], high[1], low[0], low[1]);
            upper += whole_weight(high[0] + high[1], low[0] + low[1]);
            if (xi < top) binned(xi, high[0], low[0]);
            if (xj < top && xj > -INFINITY) binned(xj, high[1], low[1]);
          },
          [&]() {
            tail += static_cast<unsigned long long>((unpack2(sum).x + unpack2(sum).y) * static_cast<float>(1ull << kFraction));
            sum = 0ull;
          });
      above += upper;
      above = warp_sum(above);
      upper = warp_sum(upper);
      tail = warp_sum(tail);
      if (lane == 0) {
        sh.above[warp] = above;
        sh.warp_mass[warp] = upper;
        sh.warp_tail[warp] = tail;
      }
      __syncthreads();
      if (warp == 0) {
        above = warp_sum(lane < kWarps ? sh.above[lane] : 0ull);
        upper = warp_sum(lane < kWarps ? sh.warp_mass[lane] : 0ull);
        tail = warp_sum(lane < kWarps ? sh.warp_tail[lane] : 0ull);
        if (lane < cs) {
          peer_store64(peer_addr(&sh.from_total[cr], lane), above);
          peer_store64(peer_addr(&sh.from_mass[cr], lane), upper);
          peer_store64(peer_addr(&sh.from_tail[cr], lane), tail);
        }
      }
      cluster_sync();
      // What top-p needs at least and at most; where that leaves two borders, by the row's mass itself.
#pragma unroll 1
      for (int exact = 0; exact < 2 && !found; ++exact) {
        if (exact) {
          cluster_sync();                 // all have read what came before
          mass_k = whole_mass();
        }
        const auto needed = [&] {         // by one warp
          if (exact) {
            if (lane == 0) sh.need = sh.need_most = part_of(top_p, mass_k, true);
            return;
          }
          const unsigned long long sure = warp_sum(lane < cs ? sh.from_total[lane] : 0ull);
          const unsigned long long known = warp_sum(lane < cs ? sh.from_mass[lane] : 0ull), rest = warp_sum(lane < cs ? sh.from_tail[lane] : 0ull);
          const unsigned long long slack = static_cast<unsigned long long>(static_cast<float>(rest) * off_by) + static_cast<unsigned long long>(v);
          if (lane == 0) {
            sh.above_all = sure;
            sh.need = part_of(top_p, known + (rest > slack ? rest - slack : 0ull), true);
          }
          if (lane == 1) sh.need_most = part_of(top_p, known + rest + slack, true);
        };
        Cross at;
        const bool there = find_cross(sh, true, needed, [&] { return sh.need > sh.above_all ? sh.need - sh.above_all : 0ull; }, at);
        above = sh.above_all;
        const unsigned long long need = sh.need, need_most = sh.need_most;
        if (need <= above) break;         // above what is sure
        if (!there) {
          settled = !guessed && from == least;   // min-p keeps less
          break;
        }
        // More than there is room for are settled only if they are all equal (logits of 16 bits).
        const bool crowd = at.in > kFew;
        uint32_t crowd_low = ~0u, crowd_high = 0u, crowd_n = 0u;
        const unsigned long long before = above + at.mass;
        // One more pass from the bin's lower end up, to the roundings of a difference and two products: the bin's values to
        // all CTAs, and the mass between it and what is sure.
        const float wide = 1e-6f * (fabsf(base) + fabsf(from));
        const float low_end = fmaxf(from, base - (static_cast<float>(at.bin) + 1.01f) / scale - wide);
        const float high_end = base - (static_cast<float>(at.bin) - 0.01f) / scale + wide;   // from here up no value is in the bin
        const auto hand = [&](float xi) {
          if (crowd) {
            const uint32_t k = float_order_key(xi);   // -0 as 0
            crowd_low = min(crowd_low, k);
            crowd_high = max(crowd_high, k);
            ++crowd_n;
            return;
          }
          const int place = static_cast<int>(at.place) + atomicAdd(&sh.few_n, 1);
          for (int r = 0; r < cs; ++r) peer_store32(peer_addr(&sh.edge.x[place], r), __float_as_uint(xi));
          sh.edge.warp[place] = static_cast<uint8_t>(warp);
        };
        unsigned long long between = 0ull;
        many_in(
            w0, w1, low_end, std::true_type{}, top, nothing,
            [&](float xi, float xj) {
              // which side of the bin a value of its neighbourhood is on, the bins say
              bool i_over = xi >= high_end, j_over = xj >= high_end;
              if (!i_over) {
                const int bin = bin_of(xi);
                if (bin == static_cast<int>(at.bin)) hand(xi);
                i_over = bin < static_cast<int>(at.bin);
              }
              if (!j_over && xj > -INFINITY) {
                const int bin = bin_of(xj);
                if (bin == static_cast<int>(at.bin)) hand(xj);
                j_over = bin < static_cast<int>(at.bin);
              }
              uint32_t high[2];
              int low[2];
              weight_pair(w, i_over ? xi : -INFINITY, j_over ? xj : -INFINITY, high[0], high[1], low[0], low[1]);
              between += whole_weight(high[0] + high[1], low[0] + low[1]);
            },
            nothing);
        between = warp_sum(between);
        if (crowd) {
          crowd_low = __reduce_min_sync(0xffffffffu, crowd_low);
          crowd_high = __reduce_max_sync(0xffffffffu, crowd_high);
          crowd_n = __reduce_add_sync(0xffffffffu, crowd_n);
          if (lane == 0) sh.warp_tail[warp] = static_cast<unsigned long long>(crowd_low) << 32 | crowd_high;
          __syncthreads();
          if (warp == 0) {
            const unsigned long long two = sh.warp_tail[lane & (kWarps - 1)];
            const uint32_t low = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(two >> 32));
            const uint32_t high = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(two));
            if (lane < cs) peer_store64(peer_addr(&sh.from_tail[cr], lane), static_cast<unsigned long long>(low) << 32 | high);
          }
        }
        cluster_sync();
        const int n = static_cast<int>(at.in);
        if (crowd) {
          const unsigned long long two = sh.from_tail[lane & (cs - 1)];
          crowd_low = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(two >> 32));
          crowd_high = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(two));
          if (crowd_low != crowd_high) break;
          if (tid == 0) {
            const unsigned long long of_one = weight(sh.w, order_key_float(crowd_low)), many = (need - before + of_one - 1) / of_one;
            sh.border = order_key_float(crowd_low);
            sh.ties = many;
            sh.reached = before + many * of_one;
          }
        } else if (tid < n) {
          sh.edge.mass[tid] = weight(sh.w, sh.edge.x[tid]);
        }
        __syncthreads();
        if (warp == 0 && !crowd) {
          // the largest key at which the mass from it up reaches what is needed: between the bin's ends, bit by bit
          uint32_t high = 0u, low = ~0u;
          for (int j = lane; j < n; j += 32) {
            const uint32_t k = float_order_key(sh.edge.x[j]);
            high = max(high, k);
            low = min(low, k);
          }
          high = __reduce_max_sync(0xffffffffu, high);
          low = __reduce_min_sync(0xffffffffu, low);
          const auto mass_from = [&](uint32_t k) {
            unsigned long long s = 0ull;
            for (int j = lane; j < n; j += 32)
              if (float_order_key(sh.edge.x[j]) >= k) s += sh.edge.mass[j];
            return before + warp_sum(s);
          };
          if (n <= 32) {                  // a lane a value
            const float xi = lane < n ? sh.edge.x[lane] : 0.0f;
            const unsigned long long mine = lane < n ? sh.edge.mass[lane] : 0ull;
            unsigned long long from_me = before;   // of its equals and those above
            for (int j = 0; j < n; ++j) {
              const unsigned long long s = __shfl_sync(0xffffffffu, mine, j);
              if (__shfl_sync(0xffffffffu, xi, j) >= xi) from_me += s;
            }
            low = __reduce_max_sync(0xffffffffu, lane < n && from_me >= need ? float_order_key(xi) : 0u);
            high = low;
          }
          while (low < high) {            // mass_from(low) reaches it
            const uint32_t mid = low + (high - low) / 2 + 1;
            if (mass_from(mid) >= need) low = mid;
            else high = mid - 1;
          }
          const unsigned long long over = low == ~0u ? before : mass_from(low + 1), of_one = weight(sh.w, order_key_float(low));
          if (lane == 0) {
            sh.border = order_key_float(low);
            // how many of its equals, at most kFew: a division in 64 bits costs as much as all of this
            unsigned long long many = static_cast<unsigned long long>(static_cast<float>(need - over) / static_cast<float>(of_one));
            while (many > 0ull && (many - 1) * of_one >= need - over) --many;
            while (many * of_one < need - over) ++many;
            sh.ties = many;
            sh.reached = over + many * of_one;
          }
        }
        __syncthreads();
        if (sh.reached >= need_most) {    // the border of all that the mass may be
          lower(sh.border, sh.ties);
          found = true;
          // what the warps keep: all above the bin, and of the bin
          if (lane == 0) sh.above[warp] += between;
          if (crowd) {
            if (lane == 0) sh.warp_count[warp] = crowd_n;
          } else if (tid < kWarps) {
            sh.warp_count[tid] = 0u;
          }
          __syncthreads();
          const int own_n = crowd ? 0 : sh.few_n;
          for (int j = tid; j < own_n; j += kThreads) {
            const int k = static_cast<int>(at.place) + j;
            const float xi = sh.edge.x[k];
            if (xi > t) atomicAdd(&sh.above[sh.edge.warp[k]], sh.edge.mass[k]);
            else if (xi == t) atomicAdd(&sh.warp_count[sh.edge.warp[k]], 1u);
          }
          __syncthreads();
        }
        if (tid == 0) sh.few_n = 0;       // read before the barrier
      }
      if (!found && (settled || !guessed)) break;
      guessed = false;
    }
    if (!found && !settled) {
      cluster_sync();
      mass_k = whole_mass();
      select(true, part_of(top_p, mass_k, true), true);
    }
    kept_known = found;
  } else if (by_p) {
    if (whole_row) mass_k = whole_mass();
    select(true, part_of(top_p, mass_k, true), true);
  }

  // kept mass and ties of the CTAs (the whole row's are known)
  if (!plain) {
    uint32_t equal = 0u;
    unsigned long long mass = 0ull;
    if (!kept_known) mass = part_kept(w0, w1, equal);
    __syncthreads();
    if (lane == 0) {
      sh.warp_mass[warp] = kept_known ? sh.above[warp] : mass;
      if (!kept_known) sh.warp_count[warp] = equal;
    }
    hand_round();
  }
  // The CTA in which the sum passes the number drawn, and the warp's part of it.
  if (warp == 0) {
    const unsigned long long of_tie = t >= w.floor ? weight(sh.w, t) : 0ull;
    unsigned long long add, left;
    unsigned long long sum = sum_parts(lane < cs ? sh.from_mass[lane] : 0ull, lane < cs ? sh.from_ties[lane] : 0u, ties, of_tie, add, left);
    const unsigned long long total = __shfl_sync(0xffffffffu, sum, 31), target = drawn(total);
    unsigned long long upto = __shfl_sync(0xffffffffu, sum - add, cr);
    const bool here = target >= upto && target < upto + __shfl_sync(0xffffffffu, add, cr);
    left = __shfl_sync(0xffffffffu, left, cr);
    int part = -1;
    if (here) {
      const unsigned long long before = upto;
      sum = before + sum_parts(lane < kWarps ? sh.warp_mass[lane] : 0ull, lane < kWarps ? sh.warp_count[lane] : 0u, left, of_tie, add, left);
      part = __ffs(__ballot_sync(0xffffffffu, target < sum)) - 1;
      upto = __shfl_sync(0xffffffffu, sum - add, part);
      left = __shfl_sync(0xffffffffu, left, part);
    }
    if (lane == 0) {
      sh.part = part;
      sh.total = total;
      sh.target = target;
      sh.upto = upto;
      sh.left = left;
      sh.of_tie = of_tie;
    }
  }
  __syncthreads();
  if (sh.part < 0) return;
  const unsigned long long target = sh.target, of_tie = sh.of_tie;
  // its sixteenths, a warp each
  const int p0 = part_begin(sh.part), p1 = part_begin(sh.part + 1);
  {
    uint32_t equal;
    const unsigned long long mass = part_kept(p0 + (p1 - p0) * warp / kWarps, p0 + (p1 - p0) * (warp + 1) / kWarps, equal);
    if (lane == 0) {
      sh.warp_mass[warp] = mass;
      sh.warp_count[warp] = equal;
    }
  }
  __syncthreads();
  if (warp != 0) return;
  unsigned long long upto, left;
  int i0, i1;
  {
    unsigned long long add;
    const unsigned long long sum = sh.upto + sum_parts(lane < kWarps ? sh.warp_mass[lane] : 0ull, lane < kWarps ? sh.warp_count[lane] : 0u,
                                                       sh.left, of_tie, add, left);
    const int part = __ffs(__ballot_sync(0xffffffffu, target < sum)) - 1;
    upto = __shfl_sync(0xffffffffu, sum - add, part);
    left = __shfl_sync(0xffffffffu, left, part);
    i0 = p0 + (p1 - p0) * part / kWarps;
    i1 = p0 + (p1 - p0) * (part + 1) / kWarps;
  }
  // and its values, 32 vectors at a time
  for (int i = i0; i < i1; i += 32) {
    unsigned long long mass = 0ull, add;
    uint32_t n = 0u;
    if (i + lane < i1) {
#pragma unroll 1
      for (int e = 0; e < W; ++e) {
        const float xi = value_at(i + lane, e);
        if (xi > t && xi >= w.floor) mass += weight(sh.w, xi);
        n += xi == t;
      }
    }
    unsigned long long mine;
    const unsigned long long sum = upto + sum_parts(mass, n, left, of_tie, add, mine);
    unsigned long long here = sum - add;
    if (target >= here && target < sum) {
#pragma unroll 1
      for (int e = 0; e < W; ++e) {
        const float xi = value_at(i + lane, e);
        unsigned long long k = 0ull;
        if (xi > t && xi >= w.floor) k = weight(sh.w, xi);
        else if (xi == t && mine > 0ull) {
          --mine;
          k = of_tie;
        }
        if (target < here + k) {
          write(xi, static_cast<uint32_t>(i + lane) * W + e - off, sh.total);
          break;
        }
        here += k;
      }
    }
    upto = __shfl_sync(0xffffffffu, sum, 31);
    const uint32_t all = __reduce_add_sync(0xffffffffu, n);
    left = left > all ? left - all : 0ull;
    if (upto > target) return;
  }
}

template <typename T, bool kHeld>
cudaError_t sample_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int64_t n, int cs, size_t shared, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};   // one bit per device; host threads may race here
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(sample_kernel<T, kHeld>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(sample_kernel<T, kHeld>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldOne);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n * cs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start before the previous grid ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaSuccess;
}

template <typename T, bool kHeld>
cudaError_t launch_sample_t(SampleArgs a, int cs, int64_t held) {
  a.held_bytes = static_cast<int>(held);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  const cudaError_t e = sample_config<T, kHeld>(cfg, attr, a.n + (a.grid == kSecond), cs, static_cast<size_t>(held) + kQueue * (kHeld ? kStaged : kRead), a.stream);
  return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, sample_kernel<T, kHeld>, a) : e;
}

// Clusters of cs CTAs that run at once, `shared` bytes each: the GPCs do not divide evenly (with two CTAs an
// SM 304, 152, 74, 36, 14 of 1, 2, 4, 8, 16).  Asked once for each device.
template <typename T>
cudaError_t clusters_at_once(int cs, bool two, int &fit) {
  static std::atomic<int> known[64][2][5];
  int dev = 0, log = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  while ((1 << log) < cs) ++log;
  std::atomic<int> &k = known[dev & 63][two][log];
  fit = k.load(std::memory_order_relaxed) - 1;
  if (fit >= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  e = sample_config<T, true>(cfg, attr, 1, cs, two ? kHeldTwo : kHeldOne, nullptr);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&fit, sample_kernel<T, true>, &cfg);
  if (e == cudaSuccess) k.store(fit + 1, std::memory_order_relaxed);
  return e;
}

constexpr int kWaves = 4, kLongRow = 32768;   // for a second grid
// As many CTAs a row as let all rows run at once, two CTAs an SM (times in us for rows of 202,048 f32 with top-p, the
// whole distribution, top-k, by CTAs a row: 32 rows 4 64, 24, 16, 8 57, 23, 15, 16 89, 34, 28; 64 rows 2 97, 34, 21, 4 77, 33,
// 20, 8 92, 41, 28; 128 rows 1 184, 67, 38, 2 142, 51, 30, 4 142, 63, 39), 1,024 values each at least; with a third more
// rows than two CTAs each have room, two each still (200 rows 198, 93, 74, one each 219, 106, 64); 16 CTAs share an SM with others
// from eight rows on, which only top-p over long rows makes up for (8 f32 rows, 16 and 8: of 50,257 26.3, 24.5 with top-p, 13.1,
// 11.6 with top-k; of 81,920 28.8, 27.6; of 100,003 28.9, 29.7; of 131,072 31.3, 32.1, top-k 13.9, 12.4; of 202,048 40.2, 43.6,
// 14.9, 13.9; 14 bf16 rows of 100,003 31.9, 31.0, of 131,072 32.8, 32.5, of 202,048 40.9, 43.3).  A share is
// held in shared memory where two CTAs' fit into an SM's (16 rows of 202,048 bf16, 8 CTAs each: 39.8, 22.2, 13.7, read
// again 40.9, 23.1, 14.1), or for the few rows that run at once with one CTA an SM.
template <typename T>
cudaError_t launch_sample_grid(const SampleArgs &a) {
  const int64_t vecs = a.v / Vec<T>::W + 2, queue = kQueue * kStaged;
  auto held = [&](int64_t cs) { return (vecs + cs - 1) / cs * 16; };   // a share is at most this
  int cs = 1, fit = 0;
  for (int next = 2; next <= kCluster && a.v / next >= 1024; next *= 2) {
    const cudaError_t e = clusters_at_once<T>(next, true, fit);
    if (e != cudaSuccess) return e;
    if (a.n > (next == 2 ? fit + fit / 3 : next == 16 && a.v < 131072 ? fit / 2 : fit)) break;
    cs = next;
  }
  if (held(cs) + queue <= kHeldTwo) return launch_sample_t<T, true>(a, cs, held(cs));
  if (held(cs) + queue <= kHeldOne) {
    const cudaError_t e = clusters_at_once<T>(cs, false, fit);
    if (e != cudaSuccess) return e;
    if (a.n <= fit) return launch_sample_t<T, true>(a, cs, held(cs));
  }
  return launch_sample_t<T, false>(a, cs, 0);
}

// Rows that fill the SMs a few times go one to a CTA; what is left then would run by itself on half of the SMs, and
// goes into a second grid, more CTAs a row, which begins as the first one's last rows end (202,048 bf16 with top-p, the whole
// distribution, top-k: 320 rows in one grid 260, 130, 71 us, in two 214, 119, 63; 400 265, 134, 78, two 239, 137, 71; 1,024
// 507, 275, 166, two 495, 279, 161).  From kLongRow on that gains more with few rows and top-p than it costs others: of
// 24,576 320 rows 54, 32, 25, two 53, 33, 25, 1,024 116, 67, 52, two 115, 72, 55; of 32,768 320 65, 38, 27, two 60, 37, 27,
// 1,024 131, 79, 56, two 134, 84, 59, 700 of f32 120, 60, 52, two 108, 63, 52; of 50,257 320 84, 54, 33, two 74, 49, 31.
template <typename T>
cudaError_t launch_sample_rows(SampleArgs a) {
  int fit = 0, pairs = 0;
  cudaError_t e = clusters_at_once<T>(1, true, fit);
  if (e == cudaSuccess) e = clusters_at_once<T>(2, true, pairs);
  if (e != cudaSuccess) return e;
  const int64_t rest = a.n % fit, first = a.n - rest;
  if (first == 0 || rest == 0 || rest > pairs || first > kWaves * fit || a.v < kLongRow) return launch_sample_grid<T>(a);
  SampleArgs b = a;
  a.grid = kFirst;
  a.n = first;
  e = launch_sample_grid<T>(a);
  if (e != cudaSuccess) return e;
  b.grid = kSecond;
  b.n = rest;
  b.logits = static_cast<const T *>(a.logits) + first * a.ld;
  b.uniforms += first;
  b.tokens += first;
  if (b.logprobs) b.logprobs += first;
  if (b.temperatures) b.temperatures += first;
  if (b.top_ks) b.top_ks += first;
  if (b.top_ps) b.top_ps += first;
  if (b.min_ps) b.min_ps += first;
  return launch_sample_grid<T>(b);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a) {
  if (a.dtype == 0) return launch_sample_rows<float>(a);
  if (a.dtype == 1) return launch_sample_rows<__half>(a);
  return launch_sample_rows<__nv_bfloat16>(a);
}

}  // namespace muse
