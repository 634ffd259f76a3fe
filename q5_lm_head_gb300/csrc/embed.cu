// Rows of a token table and the gradient by it.
//
//     out[t][j] = scale * table[token_t][j]
//     grad_table[v][j] = (accumulate ? grad_table[v][j] : 0) + scale * sum_{t: token_t = v} grad[t][j]
//
// A token outside 0..V-1 marks a padded position: a row of zeros, and nothing
// added.  The table is dense or holds the blocks of the handle's format, one row
// of the matrix a token's; products and sums in f32, rounded once to the output's
// type (sums of one token in the order of their positions).
//
// Lookup.  A warp takes 256 columns of a dense row (a lane eight), half a warp a block
// of a quantised one (a lane 16).  Bound: the dense rows' bytes (4,099 rows of 6,656
// bf16 16.3 us, 5.2 TB/s over reads and writes, most of which L2 still holds at the
// end); of blocks the unpacking, 40 million warp instructions for 16,384 rows, with the
// issue slots at 72 % and the integer pipe at 67 %: 48.9 us, 5.1 TB/s.  One token 1.4 us (2.4 with its row in HBM).
//
// Gradient.  The positions are sorted by token first, stable, so that a row of the
// table is written once, by whoever holds its sum, and the order of the sum is
// fixed.  token_order_kernel: a CTA takes a range of tokens and scans all n
// positions for them twice (counts, then places); a warp has a contiguous share of
// the positions and a counter for each token of the range, whose prefix sums are
// the places.  Every CTA reads all n tokens, from L2, which takes 27 us for 100,000
// positions of tokens spread evenly and 55 of uneven ones.
// sum_runs_kernel: a warp adds up 256 columns of a chunk of sorted positions and
// writes the runs of one token that lie inside.  A run that goes on leaves a part
// for each of its chunks; the warp that counts in last adds them up in order, so no
// warp waits for another and the bits do not depend on which that is.  Behind them
// in the same grid, a warp a row, CTAs write the zeros of rows without a token.
// Bound: HBM for a large table (16,384 positions and 202,048 x 6,656 bf16 437 us, 6.65
// TB/s, 98 % of a copy's rate), else the two kernels' chains (the order 5 us for 301
// positions, 13 for 16,384; 301 positions and 2,048 rows of 6,656 f32 19.7 us).
// Added to a table that is there, no zeros are written: 15.2, 41.5 and 154 us for 301 positions, 16,384 f16 into 32,003 x
// 1,024 f32 and into the large table, the sort first among it.
#include <atomic>

#include "common.cuh"
#include "embed_space.h"
#include "internal.h"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kLane = 8;                   // columns of a lane, of a warp's kTile

// Eight consecutive values of a lane: one access where rows lie on its size (kWide: 16
// bytes, of f32 32), two of 16 bytes for other f32 rows on 16 bytes, else value by value
// (lookup of 4,099 f32 rows of 6,656 33.9, 34.3, 88 us; gradient of 4,096 bf16 rows of 768 by
// 50,257 of f32 34.8, 38, 134 us).
template <typename T>
struct Lane8 {
  __align__(16) T v[kLane];
  __device__ __forceinline__ void load(const T *p, int access) {
    if (access == kNarrow) {
#pragma unroll
      for (int i = 0; i < kLane; ++i) v[i] = p[i];
    } else if (sizeof(T) == 2) {
      *reinterpret_cast<uint4 *>(v) = reinterpret_cast<const uint4 *>(p)[0];
    } else if (access == kWide) {
      uint32_t *r = reinterpret_cast<uint32_t *>(v);
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                   : "l"(p));
    } else {
      reinterpret_cast<uint4 *>(v)[0] = reinterpret_cast<const uint4 *>(p)[0];
      reinterpret_cast<uint4 *>(v)[sizeof(T) / 4] = reinterpret_cast<const uint4 *>(p)[1];
    }
  }
  __device__ __forceinline__ void store(T *p, int access) const {
    if (access == kNarrow) {
#pragma unroll
      for (int i = 0; i < kLane; ++i) p[i] = v[i];
    } else if (sizeof(T) == 2) {
      *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(v);
    } else if (access == kWide) {
      const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                   "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                   : "memory");
    } else {
      reinterpret_cast<uint4 *>(p)[0] = reinterpret_cast<const uint4 *>(v)[0];
      reinterpret_cast<uint4 *>(p)[1] = reinterpret_cast<const uint4 *>(v)[sizeof(T) / 4];
    }
  }
  __device__ __forceinline__ void values(float (&o)[kLane]) const {
#pragma unroll
    for (int i = 0; i < kLane; ++i) o[i] = to_float(v[i]);
  }
};

// Of memory that the grid writes too: the wide load says nothing of what it reads to the compiler (the inputs' loads
// are free to pass others), so nothing moves across this one.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int access, float (&o)[kLane]) {
  Lane8<T> r;
  asm volatile("" ::: "memory");
  r.load(p, access);
  asm volatile("" ::: "memory");
  r.values(o);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int access, const float (&o)[kLane]) {
  Lane8<T> r;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4 *>(r.v) = pack_vec(o, T{});
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) r.v[i] = o[i];
  }
  r.store(p, access);
}

// A block's 16 values of a lane of 16: eight bytes' low nibbles (one sub-block) and
// their high ones (the next).  Quants become floats as the last bits of 2^23 + q
// (a conversion instruction takes as long as all of the rest).  The products are exact
// in f32 (11 + 6 + 5 bits), so each value is rounded once.
template <bool kQ4>
struct Block16 {
  uint4 head;
  uint2 low, high;
  __device__ __forceinline__ void load(const uint8_t *block, int part) {
    head = *reinterpret_cast<const uint4 *>(block);
    low = *reinterpret_cast<const uint2 *>(block + (kQ4 ? kOffQsQ4 : kOffQs) + part * 8);
    if constexpr (!kQ4) high = *reinterpret_cast<const uint2 *>(block + kOffQh + (part & 3) * 8);
  }
  static __device__ __forceinline__ uint32_t big(uint32_t word, int byte) {   // the bits of 2^23 + that byte
    return __byte_perm(word, 0x4B000000u, 0x7650 + byte);
  }
  __device__ __forceinline__ void values(int part, float scale, float (&o)[2][kLane]) const {
    const float2 d = __half22float2(*reinterpret_cast<const __half2 *>(&head.x));
    const int s = (part >> 2) * 2;         // the first of the two sub-blocks
    // scales and mins of four sub-blocks, a byte each: 0..3, or 4..7 (4 bits there, 2 above those of the first)
    const bool late = s >= 4;
    const uint32_t sc = late ? (head.w & 0x0F0F0F0Fu) | ((head.y >> 2) & 0x30303030u) : head.y & 0x3F3F3F3Fu;
    const uint32_t mn = late ? ((head.w >> 4) & 0x0F0F0F0Fu) | ((head.z >> 2) & 0x30303030u) : head.z & 0x3F3F3F3Fu;
    const unsigned long long off = pack2(-8388608.0f, -8388608.0f), by = pack2(scale, scale);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float ds = d.x * (__uint_as_float(big(sc, (s & 2) + h)) - 8388608.0f);
      const float dm = -(d.y * (__uint_as_float(big(mn, (s & 2) + h)) - 8388608.0f));
      uint32_t q[2] = {(low.x >> (4 * h)) & 0x0F0F0F0Fu, (low.y >> (4 * h)) & 0x0F0F0F0Fu};
      if constexpr (!kQ4) {                // bit s + h of each byte, to bit 4
        q[0] |= __funnelshift_l(high.x, high.x, 4 - s - h) & 0x10101010u;
        q[1] |= __funnelshift_l(high.y, high.y, 4 - s - h) & 0x10101010u;
      }
      const unsigned long long ds2 = pack2(ds, ds), dm2 = pack2(dm, dm);
#pragma unroll
      for (int i = 0; i < kLane; i += 2) {
        const unsigned long long x =
            add2(pack2(__uint_as_float(big(q[i >> 2], i & 3)), __uint_as_float(big(q[i >> 2], (i & 3) + 1))), off);
        const float2 r = unpack2(mul2(fma2(ds2, x, dm2), by));
        o[h][i] = r.x;
        o[h][i + 1] = r.y;
      }
    }
  }
};

// Lookup in a dense table.  A warp takes kTiles tiles, all of whose loads are under way before the first is used.
template <typename TT, typename TO, int kTiles>
__global__ void __launch_bounds__(256) embed_dense_kernel(const EmbedArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the tokens are complete
  const int lane = threadIdx.x & 31, tiles = a.k / kTile;
  const int64_t items = a.n * tiles, step = static_cast<int64_t>(gridDim.x) * 8 * kTiles;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kTiles; i < items; i += step) {
    int64_t t = i / tiles;
    int tile = static_cast<int>(i - t * tiles);
    Lane8<TT> raw[kTiles];
    int64_t to[kTiles];
    bool ok[kTiles];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      const bool in = i + j < items;
      to[j] = in ? t * a.out_ld + tile * kTile + lane * kLane : -1;
      const int64_t tok = in ? a.tokens[t] : -1;
      ok[j] = tok >= 0 && tok < a.v;
      const int64_t from = ok[j] ? tok : 0;             // a padded position reads the first row and leaves it
      raw[j].load(static_cast<const TT *>(a.table) + from * a.table_ld + tile * kTile + lane * kLane, a.access_in);
      if (++tile == tiles) {
        tile = 0;
        ++t;
      }
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      float o[kLane];
      raw[j].values(o);
#pragma unroll
      for (int e = 0; e < kLane; ++e) o[e] = ok[j] ? o[e] * a.scale : 0.0f;
      if (to[j] >= 0) store8(static_cast<TO *>(a.out) + to[j], a.access_out, o);
    }
  }
}

// Lookup in a table of blocks.  Half a warp takes a block; a CTA kRounds * 16 of them
// that follow one another, all loads of a warp under way before the first is used.
template <bool kQ4, typename TO, int kRounds>
__global__ void __launch_bounds__(256) embed_blocks_kernel(const EmbedArgs a) {
  constexpr int kBytes = kQ4 ? kBlockBytesQ4 : kBlockBytes;
  const int part = threadIdx.x & 15, tiles = a.k / kTile;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (16 * kRounds);
  int64_t t = first / tiles;
  int tile = static_cast<int>(first - t * tiles) + (threadIdx.x >> 4);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the tokens are complete
  Block16<kQ4> raw[kRounds];
  int64_t to[kRounds];
  bool ok[kRounds];
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    while (tile >= tiles) {
      tile -= tiles;
      ++t;
    }
    const int64_t tok = t < a.n ? a.tokens[t] : -1;
    ok[j] = tok >= 0 && tok < a.v;
    to[j] = t < a.n ? t * a.out_ld + tile * kTile + (part >> 2) * 64 + (part & 3) * 8 : -1;
    if (ok[j]) raw[j].load(static_cast<const uint8_t *>(a.table) + (tok * tiles + tile) * kBytes, part);
    tile += 16;
  }
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    float o[2][kLane] = {};
    if (ok[j]) raw[j].values(part, a.scale, o);
    if (to[j] >= 0) {
      store8(static_cast<TO *>(a.out) + to[j], a.access_out, o[0]);
      store8(static_cast<TO *>(a.out) + to[j] + 32, a.access_out, o[1]);
    }
  }
}

template <typename A>
cudaError_t launch_after(void (*kernel)(A), int64_t grid, int threads, size_t shared, cudaStream_t stream, A a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start before the previous grid ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Four tiles a warp from 24 warps of one tile an SM on, else one (times in us by rows of 6,656 bf16, one tile and
// four: 16 1.47, 1.62; 128 1.73, 1.71; 256 2.40, 2.07; 1,024 6.5, 4.6; 16,384 91, 69).
template <typename TT, typename TO>
cudaError_t launch_embed_dense(const EmbedArgs &a) {
  const int64_t items = a.n * (a.k / kTile), most = int64_t{1} << 30;
  const bool many = items >= 24 * static_cast<int64_t>(a.num_sms);
  const int64_t blocks = (items + (many ? 31 : 7)) / (many ? 32 : 8);
  void (*kernel)(EmbedArgs) = many ? embed_dense_kernel<TT, TO, 4> : embed_dense_kernel<TT, TO, 1>;
  return launch_after(kernel, blocks < most ? blocks : most, 256, 0, a.stream, a);
}
// Four rounds of blocks a warp from 256 blocks an SM on, else one (Q5_K rows of 6,656 to bf16: 64 1.47, 2.65; 512
// 2.58, 3.26; 1,024 3.95, 4.04; 4,099 14.9, 14.7; 16,384 54, 51).
template <bool kQ4, typename TO>
cudaError_t launch_embed_blocks(const EmbedArgs &a) {
  const int64_t items = a.n * (a.k / kTile);
  const bool many = items >= 256 * static_cast<int64_t>(a.num_sms);
  const int64_t blocks = (items + (many ? 63 : 15)) / (many ? 64 : 16);
  void (*kernel)(EmbedArgs) = many ? embed_blocks_kernel<kQ4, TO, 4> : embed_blocks_kernel<kQ4, TO, 1>;
  return launch_after(kernel, blocks, 256, 0, a.stream, a);
}

template <typename TO>
cudaError_t launch_embed_to(const EmbedArgs &a) {
  switch (a.table_type) {
    case 0: return launch_embed_dense<float, TO>(a);
    case 1: return launch_embed_dense<__half, TO>(a);
    case 2: return launch_embed_dense<__nv_bfloat16, TO>(a);
    default: return a.q4 ? launch_embed_blocks<true, TO>(a) : launch_embed_blocks<false, TO>(a);
  }
}

// ---------------------------------------------------------------- gradient by the table
constexpr int kOrderThreads = 1024;
constexpr int kOrderWarps = kOrderThreads / 32;
constexpr int kMaxRange = 1536;            // tokens of a CTA: 34 words each, 204 KB
constexpr int kUnroll = 16;                // positions of a lane in flight; up to 16,384 positions are read once

// One scan or two, as n allows, of all positions by every CTA; latency: loads, counters in shared memory, the prefix
// sums of 32 warps' counters.

__global__ void __launch_bounds__(kOrderThreads) token_order_kernel(const EmbedBackwardArgs a) {
  extern __shared__ int s_count[];         // [warps][range]: counts, then places; [range] runs' first places, [range] their ends
  __shared__ int s_warp[kOrderWarps], s_below[kOrderWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, range = a.range;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * range;
  const int size = static_cast<int>(a.v - lo < range ? a.v - lo : range);
  for (int i = tid; i < kOrderWarps * range; i += kOrderThreads) s_count[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the tokens are complete
  __syncthreads();

  // this warp's positions, a multiple of 32 of them
  const int64_t share = (a.n + kOrderThreads - 1) / kOrderThreads * 32;
  const int64_t p0 = warp * share, p1 = p0 + share < a.n ? p0 + share : a.n;
  const bool once = share <= 32 * kUnroll;   // then the second scan has its tokens still
  const uint32_t first = static_cast<uint32_t>(lo);
  int *mine = s_count + warp * range, *s_first = s_count + kOrderWarps * range, *s_end = s_first + range;
  int below = 0;
  uint32_t tok[kUnroll];                   // a padded position is at least 2^31, beyond every range
  auto fetch = [&](int64_t p) {
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) tok[j] = p + j * 32 + lane < p1 ? static_cast<uint32_t>(a.tokens[p + j * 32 + lane]) : ~0u;
  };
  for (int64_t p = p0; p < p1; p += 32 * kUnroll) {
    fetch(p);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      below += tok[j] < first;
      if (tok[j] - first < static_cast<uint32_t>(size)) atomicAdd(mine + (tok[j] - first), 1);
    }
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) s_below[warp] = below;
  __syncthreads();

  // places: tokens in order, a token's warps in order
  constexpr int kEach = (kMaxRange + kOrderThreads - 1) / kOrderThreads;
  int total[kEach], sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int t = tid * kEach + e;
    total[e] = 0;
    if (t < size) {
#pragma unroll
      for (int w = 0; w < kOrderWarps; ++w) total[e] += s_count[w * range + t];
    }
    sum += total[e];
  }
  int upto = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int at = upto - sum, all = 0;
  for (int w = 0; w < kOrderWarps; ++w) {
    if (w < warp) at += s_warp[w];
    at += s_below[w];
    all += s_warp[w] + s_below[w];
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int t = tid * kEach + e;
    if (t < size) {
      s_first[t] = at;
      s_end[t] = at + total[e];
      if (total[e] == 0) continue;         // its places are of no use
#pragma unroll
      for (int half = 0; half < kOrderWarps; half += 16) {
        int c[16];
#pragma unroll
        for (int w = 0; w < 16; ++w) c[w] = s_count[(half + w) * range + t];
#pragma unroll
        for (int w = 0; w < 16; ++w) {
          s_count[(half + w) * range + t] = at;
          at += c[w];
        }
      }
    }
  }
  if (tid == 0 && blockIdx.x == gridDim.x - 1) *a.count = all;
  __syncthreads();

  // which rows have a token, and counters of nothing
  for (int t = warp * 32; t < size; t += kOrderThreads) {
    const uint32_t used = __ballot_sync(0xffffffffu, t + lane < size && s_end[t + lane] > s_first[t + lane]);
    if (lane == 0) a.used[(lo + t) / 32] = used;
  }
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kOrderThreads + tid; i < a.done_n; i += static_cast<int64_t>(gridDim.x) * kOrderThreads) a.done[i] = 0;

  __syncthreads();                         // a place is moved on below
  for (int64_t p = p0; p < p1; p += 32 * kUnroll) {
    if (!once) fetch(p);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t t = tok[j] - first;
      const bool in = t < static_cast<uint32_t>(size);
      const uint32_t some = __ballot_sync(0xffffffffu, in);
      if (some == 0u) continue;
      int place = 0;
      uint32_t same = 0u;
      if (in) {
        same = __match_any_sync(some, t);
        place = mine[t] + __popc(same & ((1u << lane) - 1u));
      }
      __syncwarp();
      if (in) {
        if (lane == 31 - __clz(same)) mine[t] = place + 1;
        a.order[place] = static_cast<int>(p + j * 32 + lane);
        a.sorted[place] = static_cast<int>(tok[j]);
        a.span[place] = make_int2(s_first[t], s_end[t]);
      }
      __syncwarp();
    }
  }
}

template <typename TO>
__device__ __forceinline__ void write_sum(const EmbedBackwardArgs &a, int64_t tok, int col, const float (&s)[kLane]) {
  TO *p = static_cast<TO *>(a.grad_table) + tok * a.table_ld + col;
  float o[kLane];
  if (a.accumulate) {
    load8(p, a.access_out, o);
#pragma unroll
    for (int i = 0; i < kLane; ++i) o[i] = fmaf(s[i], a.scale, o[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) o[i] = s[i] * a.scale;
  }
  store8(p, a.access_out, o);
}

constexpr int kGroup = 32, kManyParts = 64;   // chunks of a group, parts that are joined by groups

// After a chunk's part of a run of several chunks is stored: the last warp to come adds the parts up, in order.  From
// kManyParts on the chunks of a group are joined first, its sum in place of its first part (16,384 times one token,
// 1,024 columns: 57 us, all parts by one warp 161).  Counters: chunks that the run holds to the end count no
// other one, so a group takes its first chunk's, the run the one it begins in, whose group then takes the next.
template <typename TO>
__device__ __forceinline__ void join_run(const EmbedBackwardArgs &a, int2 span, int tok, int chunk, int tile) {
  const int lane = threadIdx.x & 31, tiles = a.k / kTile, col = tile * kTile + lane * kLane;
  const int from = span.x / a.chunk, last = (span.y - 1) / a.chunk;
  const int group = chunk / kGroup * kGroup, g0 = group > from ? group : from, g1 = group + kGroup - 1 < last ? group + kGroup - 1 : last;
  const bool many = last - from >= kManyParts;
  // first of all a group's parts, where it has two or more
  int first = g0, next = g0 + 1, step = 1, more = g1 - g0, counter = g0 == from ? from + 1 : g0;
  for (bool whole = !many || more == 0;; whole = true) {
    if (whole) {
      first = counter = from;
      next = many ? from / kGroup * kGroup + kGroup : from + 1;
      step = many ? kGroup : 1;
      more = many ? last / kGroup - from / kGroup : last - from;
    }
    int came = 0;
    __syncwarp();                          // lane 0 counts for the stores of all
    __threadfence();
    if (lane == 0) came = atomicAdd(a.done + (static_cast<int64_t>(counter) * tiles + tile), 1);
    if (__shfl_sync(0xffffffffu, came, 0) != more) return;
    __threadfence();                       // all parts are there, for lane 0
    __syncwarp();                          // and so for the others
    float *to = a.part + (static_cast<int64_t>(first * 2 + (first == from)) * a.k + col);
    const float *part = a.part + (static_cast<int64_t>(next) * 2 * a.k + col);
    const int64_t far = static_cast<int64_t>(step) * 2 * a.k;
    float sum[kLane];
    load8(to, kWide, sum);
    constexpr int kParts = 4;              // in flight
    for (int c = 0; c < more; c += kParts, part += kParts * far) {
      float v[kParts][kLane];
#pragma unroll
      for (int u = 0; u < kParts; ++u)
        if (c + u < more) load8(part + u * far, kWide, v[u]);
#pragma unroll
      for (int u = 0; u < kParts; ++u)
        if (c + u < more) {
#pragma unroll
          for (int i = 0; i < kLane; ++i) sum[i] += v[u][i];
        }
    }
    if (whole) {
      write_sum<TO>(a, tok, col, sum);
      return;
    }
    store8(to, kWide, sum);
  }
}

template <typename TG, typename TO>
__global__ void __launch_bounds__(256, 3) sum_runs_kernel(const __grid_constant__ EmbedBackwardArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tiles = a.k / kTile;
  if (blockIdx.x >= a.sum_blocks) {        // rows without a token
    const int64_t item = static_cast<int64_t>(blockIdx.x - a.sum_blocks) * 8 + warp, row = item / a.zero_parts;
    if (row >= a.v || ((a.used[row / 32] >> (row % 32)) & 1u)) return;
    const int part = static_cast<int>(item - row * a.zero_parts);
    const float o[kLane] = {};
    TO *p = static_cast<TO *>(a.grad_table) + row * a.table_ld + lane * kLane;
    const int end = tiles * (part + 1) / a.zero_parts;
    for (int j = tiles * part / a.zero_parts; j < end; ++j) store8(p + j * kTile, a.access_out, o);
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  const int64_t chunk = item / tiles;
  const int tile = static_cast<int>(item - chunk * tiles), col = tile * kTile + lane * kLane;
  // all that it needs to know at once: what lies behind the last position is there, but of no use
  const int64_t j0 = chunk * a.chunk, all = j0 + a.chunk < a.n ? j0 + a.chunk : a.n;
  if (j0 >= a.n) return;
  const int count = *a.count;
  int pos = j0 + lane < all ? a.order[j0 + lane] : 0, tok = j0 + lane < all ? a.sorted[j0 + lane] : -1;
  const int2 span0 = a.span[j0];
  if (j0 >= count) return;
  const int64_t j1 = all < count ? all : count;
  const int2 span1 = a.span[j1 - 1];
  const bool begun = span0.x < j0, goes_on = span1.y > j1;   // runs that other chunks hold a part of
  const TG *g = static_cast<const TG *>(a.grad) + col;

  float s[kLane];
#pragma unroll
  for (int i = 0; i < kLane; ++i) s[i] = 0.0f;
  int run = -1;
  bool first = true;                       // the run that the chunk begins with
  auto put = [&](bool last) {              // a part of a run of several chunks: its first chunk's second one, the others' first ones
    const bool head = first && begun;
    if (head || (last && goes_on)) store8(a.part + (chunk * 2 + !head) * a.k + col, kWide, s);
    else write_sum<TO>(a, run, col, s);
  };
  constexpr int kFlight = sizeof(TG) == 4 ? 4 : 8;   // positions in flight: 32 registers
  for (int64_t j = j0; j < j1; j += 32) {
    const int many = static_cast<int>(j1 - j < 32 ? j1 - j : 32);
    if (j > j0) {
      pos = lane < many ? a.order[j + lane] : 0;
      tok = lane < many ? a.sorted[j + lane] : -1;
    }
    for (int b = 0; b < many; b += kFlight) {
      Lane8<TG> raw[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        if (b + u < many) raw[u].load(g + static_cast<int64_t>(__shfl_sync(0xffffffffu, pos, b + u)) * a.grad_ld, a.access_in);
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        if (b + u < many) {
          const int t = __shfl_sync(0xffffffffu, tok, b + u);
          if (t != run) {
            if (run >= 0) {
              put(false);
              first = false;
#pragma unroll
              for (int i = 0; i < kLane; ++i) s[i] = 0.0f;
            }
            run = t;
          }
          float v[kLane];
          raw[u].values(v);
#pragma unroll
          for (int i = 0; i < kLane; ++i) s[i] += v[i];
        }
    }
  }
  put(true);
  if (begun) join_run<TO>(a, span0, a.sorted[j0], static_cast<int>(chunk), tile);
  if (goes_on && !(first && begun)) join_run<TO>(a, span1, run, static_cast<int>(chunk), tile);
}

template <typename TG, typename TO>
cudaError_t launch_sum_runs(EmbedBackwardArgs a, int64_t chunks) {
  a.sum_blocks = static_cast<unsigned>((chunks * (a.k / kTile) + 7) / 8);
  // a warp zeroes a row, or a part of it where there are few (1,024 rows of 6,656 bf16, parts 1 17.5, 4 16.7 us; 50,257
  // rows of 768 f32 parts 1 34.9, 2 43)
  const int tiles = a.k / kTile;
  a.zero_parts = 1;
  while (a.zero_parts < tiles && a.v * a.zero_parts < 48 * static_cast<int64_t>(a.num_sms)) a.zero_parts *= 2;
  const int64_t zero_blocks = a.accumulate ? 0 : (a.v * a.zero_parts + 7) / 8;
  return launch_after(sum_runs_kernel<TG, TO>, a.sum_blocks + zero_blocks, 256, 0, a.stream, a);
}

template <typename TO>
cudaError_t launch_sum_runs_to(const EmbedBackwardArgs &a, int64_t chunks) {
  if (a.dtype == 0) return launch_sum_runs<float, TO>(a, chunks);
  if (a.dtype == 1) return launch_sum_runs<__half, TO>(a, chunks);
  return launch_sum_runs<__nv_bfloat16, TO>(a, chunks);
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs &a) {
  if (a.out_dtype == 0) return launch_embed_to<float>(a);
  if (a.out_dtype == 1) return launch_embed_to<__half>(a);
  return launch_embed_to<__nv_bfloat16>(a);
}

size_t embed_backward_bytes(int64_t n, int64_t v, int k, int num_sms) { return backward_space(n, v, k, num_sms).bytes; }

cudaError_t launch_embed_backward(EmbedBackwardArgs a, void *workspace) {
  const BackwardSpace s = backward_space(a.n, a.v, a.k, a.num_sms);
  uint8_t *w = space_base(workspace);
  a.count = reinterpret_cast<int *>(w);
  a.order = reinterpret_cast<int *>(w + s.order);
  a.sorted = reinterpret_cast<int *>(w + s.sorted);
  a.span = reinterpret_cast<int2 *>(w + s.span);
  a.used = reinterpret_cast<uint32_t *>(w + s.used);
  a.done = reinterpret_cast<int *>(w + s.done);
  a.done_n = s.chunks * (a.k / kTile);
  a.part = reinterpret_cast<float *>(w + s.part);
  a.chunk = static_cast<int>(s.chunk);
  // tokens of a CTA: a share of them, in whole words of `used`
  const int64_t range = (a.v + a.num_sms - 1) / a.num_sms;
  a.range = static_cast<int>(range < kMaxRange ? (range + 31) / 32 * 32 : kMaxRange);
  static std::atomic<unsigned long long> configured{0};   // one bit per device; host threads may race here
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(token_order_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(int) * (kOrderWarps + 2) * kMaxRange));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  e = launch_after(token_order_kernel, (a.v + a.range - 1) / a.range, kOrderThreads, sizeof(int) * (kOrderWarps + 2) * a.range,
                   a.stream, a);
  if (e != cudaSuccess) return e;
  if (a.out_dtype == 0) return launch_sum_runs_to<float>(a, s.chunks);
  if (a.out_dtype == 1) return launch_sum_runs_to<__half>(a, s.chunks);
  return launch_sum_runs_to<__nv_bfloat16>(a, s.chunks);
}

}  // namespace muse
