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
// Lookup.  A warp takes 256 columns of a row, one block of a quantised table: a
// lane's eight consecutive columns lie in one sub-block and are one or two 16-byte
// vectors of the output.
//
// Gradient.  The positions are sorted by token first, stable, so that a row of the
// table is written once, by whoever holds its sum, and the order of the sum is
// fixed.  token_order_kernel: a CTA takes a range of tokens and scans all n
// positions for them twice (counts, then places); a warp has a contiguous share of
// the positions and a counter for each token of the range, whose prefix sums are
// the places.  Reading n tokens in every CTA costs n * 4 bytes of L2 against the
// n * k * 2 bytes of the gradient divided by the number of CTAs, 2 % at most.  It
// also writes the zeros of rows without a token, whose counts it has.
// sum_runs_kernel: a warp adds up 256 columns of a chunk of sorted positions and
// writes the runs of one token that lie inside; a run that goes on leaves a part
// for each chunk, which join_runs_kernel adds up in order.
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kTile = 256;                 // columns of a warp: a block
constexpr int kLane = 8;                   // of a lane

template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, float (&o)[kLane]) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p)), b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
      float lo[4], hi[4];
      unpack(a, lo, T{});
      unpack(b, hi, T{});
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = lo[i];
        o[i + 4] = hi[i];
      }
    } else {
      unpack(__ldcs(reinterpret_cast<const uint4 *>(p)), o, T{});
    }
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) o[i] = to_float(p[i]);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, bool vec, const float (&o)[kLane]) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      float4 *q = reinterpret_cast<float4 *>(p);
      q[0] = make_float4(o[0], o[1], o[2], o[3]);
      q[1] = make_float4(o[4], o[5], o[6], o[7]);
    } else {
      *reinterpret_cast<uint4 *>(p) = pack_vec(o, T{});
    }
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) p[i] = from_float<T>(o[i]);
  }
}

// Values 8 lane .. 8 lane + 7 of a block: one sub-block's.  The products are exact in
// f32 (11 + 6 + 5 bits), so each value is rounded once.
template <bool kQ4>
__device__ __forceinline__ void block8(const uint8_t *block, int lane, float (&o)[kLane]) {
  const uint4 head = *reinterpret_cast<const uint4 *>(block);
  const float2 d = __half22float2(*reinterpret_cast<const __half2 *>(&head.x));
  const int s = lane >> 2, at = (lane & 3) * 8;
  int sc, m;
  q5k_scale_min(head.y, head.z, head.w, s, sc, m);
  const uint2 low = *reinterpret_cast<const uint2 *>(block + (kQ4 ? kOffQsQ4 : kOffQs) + (s >> 1) * 32 + at);
  const uint32_t shift = (s & 1) * 4;
  uint32_t q[2] = {(low.x >> shift) & 0x0F0F0F0Fu, (low.y >> shift) & 0x0F0F0F0Fu};
  if constexpr (!kQ4) {
    const uint2 high = *reinterpret_cast<const uint2 *>(block + kOffQh + at);
    q[0] |= ((high.x >> s) & 0x01010101u) << 4;
    q[1] |= ((high.y >> s) & 0x01010101u) << 4;
  }
  const float ds = d.x * static_cast<float>(sc), dm = d.y * static_cast<float>(m);
#pragma unroll
  for (int i = 0; i < kLane; ++i) o[i] = fmaf(ds, static_cast<float>((q[i >> 2] >> (8 * (i & 3))) & 255u), -dm);
}

enum class Table { Dense, Q5, Q4 };

template <Table kTable, typename TT, typename TO>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the tokens are complete
  const int lane = threadIdx.x & 31, tiles = a.k / kTile;
  const int64_t items = a.n * tiles, step = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5); i < items; i += step) {
    const int64_t t = i / tiles;
    const int tile = static_cast<int>(i - t * tiles);
    const int64_t tok = a.tokens[t];
    float o[kLane];
#pragma unroll
    for (int j = 0; j < kLane; ++j) o[j] = 0.0f;
    if (tok >= 0 && tok < a.v) {
      if constexpr (kTable == Table::Dense) {
        load8(static_cast<const TT *>(a.table) + tok * a.table_ld + tile * kTile + lane * kLane, a.vec_in, o);
      } else {
        constexpr int kBytes = kTable == Table::Q4 ? kBlockBytesQ4 : kBlockBytes;
        block8<kTable == Table::Q4>(static_cast<const uint8_t *>(a.table) + (tok * tiles + tile) * kBytes, lane, o);
      }
#pragma unroll
      for (int j = 0; j < kLane; ++j) o[j] *= a.scale;
    }
    store8(static_cast<TO *>(a.out) + t * a.out_ld + tile * kTile + lane * kLane, a.vec_out, o);
  }
}

template <Table kTable, typename TT, typename TO>
cudaError_t launch_embed_t(const EmbedArgs &a) {
  const int64_t items = a.n * (a.k / kTile), blocks = (items + 7) / 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < (int64_t{1} << 30) ? blocks : int64_t{1} << 30));
  cfg.blockDim = dim3(256);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start before the previous grid ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, embed_kernel<kTable, TT, TO>, a);
}

template <Table kTable, typename TT>
cudaError_t launch_embed_out(const EmbedArgs &a) {
  if (a.out_dtype == 0) return launch_embed_t<kTable, TT, float>(a);
  if (a.out_dtype == 1) return launch_embed_t<kTable, TT, __half>(a);
  return launch_embed_t<kTable, TT, __nv_bfloat16>(a);
}

// ---------------------------------------------------------------- gradient by the table
constexpr int kOrderThreads = 512;
constexpr int kOrderWarps = kOrderThreads / 32;
constexpr int kMaxRange = 1536;            // tokens of a CTA: 16 counters each, 96 KB
constexpr int kUnroll = 8;                 // positions of a lane in flight

// Zeros of a row of the table by a warp.
template <typename TO>
__device__ __forceinline__ void zero_row(TO *row, int k, bool vec, int lane) {
  const float o[kLane] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = lane * kLane; j < k; j += kTile) store8(row + j, vec, o);
}

template <typename TO>
__global__ void __launch_bounds__(kOrderThreads) token_order_kernel(const EmbedBackwardArgs a) {
  extern __shared__ int s_count[];         // [warps][range]: counts, then places
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
  int *mine = s_count + warp * range;
  int below = 0;
  for (int64_t p = p0; p < p1; p += 32 * kUnroll) {
    int64_t tok[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) tok[j] = p + j * 32 + lane < p1 ? a.tokens[p + j * 32 + lane] : -1;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      below += tok[j] >= 0 && tok[j] < lo;
      if (tok[j] >= lo && tok[j] < lo + size) atomicAdd(mine + (tok[j] - lo), 1);
    }
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) s_below[warp] = below;
  __syncthreads();

  // places: tokens in order, a token's warps in order
  constexpr int kEach = kMaxRange / kOrderThreads;
  int total[kEach], sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int t = tid * kEach + e;
    total[e] = 0;
    if (t < size)
      for (int w = 0; w < kOrderWarps; ++w) total[e] += s_count[w * range + t];
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
      for (int w = 0; w < kOrderWarps; ++w) {
        const int c = s_count[w * range + t];
        s_count[w * range + t] = total[e] == 0 ? -1 : at;   // -1: a row without a token
        at += c;
      }
    }
  }
  if (tid == 0 && blockIdx.x == gridDim.x - 1) *a.count = all;
  __syncthreads();

  if (!a.accumulate)
    for (int t = warp; t < size; t += kOrderWarps)
      if (s_count[t] < 0) zero_row(static_cast<TO *>(a.grad_table) + (lo + t) * a.table_ld, a.k, a.vec_out, lane);

  __syncthreads();                         // a place is moved on below
  for (int64_t p = p0; p < p1; p += 32 * kUnroll) {
    int64_t tok[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) tok[j] = p + j * 32 + lane < p1 ? a.tokens[p + j * 32 + lane] : -1;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const bool in = tok[j] >= lo && tok[j] < lo + size;
      const uint32_t some = __ballot_sync(0xffffffffu, in);
      if (some == 0u) continue;
      int place = 0;
      uint32_t same = 0u;
      if (in) {
        same = __match_any_sync(some, static_cast<int>(tok[j] - lo));
        place = mine[tok[j] - lo] + __popc(same & ((1u << lane) - 1u));
      }
      __syncwarp();
      if (in) {
        if (lane == 31 - __clz(same)) mine[tok[j] - lo] = place + 1;
        a.order[place] = static_cast<int>(p + j * 32 + lane);
        a.sorted[place] = static_cast<int>(tok[j]);
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
    load8(p, a.vec_out, o);
#pragma unroll
    for (int i = 0; i < kLane; ++i) o[i] = fmaf(s[i], a.scale, o[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) o[i] = s[i] * a.scale;
  }
  store8(p, a.vec_out, o);
}

template <typename TG, typename TO>
__global__ void __launch_bounds__(256) sum_runs_kernel(const EmbedBackwardArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, tiles = a.k / kTile;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t chunk = item / tiles;
  const int col = static_cast<int>(item - chunk * tiles) * kTile + lane * kLane;
  const int count = *a.count;
  const int64_t j0 = chunk * a.chunk;
  if (j0 >= count) return;
  const int64_t j1 = j0 + a.chunk < count ? j0 + a.chunk : count;
  const int before = j0 > 0 ? a.sorted[j0 - 1] : -1, after = j1 < count ? a.sorted[j1] : -1;
  const TG *g = static_cast<const TG *>(a.grad) + col;
  float *part = a.part + chunk * 2 * a.k + col;

  float s[kLane];
#pragma unroll
  for (int i = 0; i < kLane; ++i) s[i] = 0.0f;
  int run = -1;
  bool first = true;                       // the run that the chunk begins with
  auto put = [&](int tok, bool last) {
    if (first && tok == before) store8(part, true, s);
    else if (last && tok == after) store8(part + a.k, true, s);
    else write_sum<TO>(a, tok, col, s);
  };
  for (int64_t j = j0; j < j1; j += 32) {
    const int many = static_cast<int>(j1 - j < 32 ? j1 - j : 32);
    const int pos = lane < many ? a.order[j + lane] : 0, tok = lane < many ? a.sorted[j + lane] : -1;
    for (int b = 0; b < many; b += kUnroll) {
      float v[kUnroll][kLane];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (b + u < many) load8(g + static_cast<int64_t>(__shfl_sync(0xffffffffu, pos, b + u)) * a.grad_ld, a.vec_in, v[u]);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (b + u < many) {
          const int t = __shfl_sync(0xffffffffu, tok, b + u);
          if (t != run) {
            if (run >= 0) {
              put(run, false);
              first = false;
#pragma unroll
              for (int i = 0; i < kLane; ++i) s[i] = 0.0f;
            }
            run = t;
          }
#pragma unroll
          for (int i = 0; i < kLane; ++i) s[i] += v[u][i];
        }
    }
  }
  put(run, true);
}

// The runs that chunks share: by the chunk in which one begins.
template <typename TO>
__global__ void __launch_bounds__(256) join_runs_kernel(const EmbedBackwardArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, tiles = a.k / kTile;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t chunk = item / tiles;
  const int col = static_cast<int>(item - chunk * tiles) * kTile + lane * kLane;
  const int count = *a.count;
  const int64_t j0 = chunk * a.chunk, j1 = j0 + a.chunk;
  if (j1 >= count) return;
  const int tok = a.sorted[j1];
  if (a.sorted[j1 - 1] != tok) return;                                     // nothing goes on
  if (j0 > 0 && a.sorted[j0] == tok && a.sorted[j0 - 1] == tok) return;    // begun before
  // chunks after this one that the run reaches into: until one has another token at its end
  int64_t more = 1;
  for (;; more += 32) {
    const int64_t end = (chunk + more + lane + 1) * a.chunk;
    const uint32_t stop = __ballot_sync(0xffffffffu, end >= count || a.sorted[end] != tok);
    if (stop) {
      more += __ffs(stop) - 1;
      break;
    }
  }
  const float *part = a.part + chunk * 2 * a.k + col;
  float s[kLane];
  load8(part + a.k, true, s);
  for (int64_t c = 1; c <= more; c += kUnroll) {
    float v[kUnroll][kLane];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (c + u <= more) load8(part + (c + u) * 2 * a.k, true, v[u]);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (c + u <= more) {
#pragma unroll
        for (int i = 0; i < kLane; ++i) s[i] += v[u][i];
      }
  }
  write_sum<TO>(a, tok, col, s);
}

template <typename... Args>
cudaError_t launch_after(void (*kernel)(Args...), int64_t grid, int threads, size_t shared, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Sorted positions of a chunk: at most 1,024 chunks, whose parts stay small beside the gradient.
int64_t chunk_of(int64_t n) {
  int64_t c = 16;
  while (c * 1024 < n) c *= 2;
  return c;
}

template <typename TO>
cudaError_t launch_embed_backward_t(EmbedBackwardArgs a) {
  int64_t range = (a.v + a.num_sms - 1) / a.num_sms;
  a.range = static_cast<int>(range < kMaxRange ? range : kMaxRange);
  const size_t shared = sizeof(int) * kOrderWarps * a.range;
  static std::atomic<unsigned long long> configured{0};   // one bit per device; host threads may race here
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(token_order_kernel<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(int) * kOrderWarps * kMaxRange));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  e = launch_after(token_order_kernel<TO>, (a.v + a.range - 1) / a.range, kOrderThreads, shared, a.stream, a);
  if (e != cudaSuccess || a.n == 0) return e;
  const int64_t chunks = (a.n + a.chunk - 1) / a.chunk, grid = (chunks * (a.k / kTile) + 7) / 8;
  if (a.dtype == 0) e = launch_after(sum_runs_kernel<float, TO>, grid, 256, 0, a.stream, a);
  else if (a.dtype == 1) e = launch_after(sum_runs_kernel<__half, TO>, grid, 256, 0, a.stream, a);
  else e = launch_after(sum_runs_kernel<__nv_bfloat16, TO>, grid, 256, 0, a.stream, a);
  if (e != cudaSuccess || chunks == 1) return e;
  return launch_after(join_runs_kernel<TO>, grid, 256, 0, a.stream, a);
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs &a) {
  switch (a.table_type) {
    case 0: return launch_embed_out<Table::Dense, float>(a);
    case 1: return launch_embed_out<Table::Dense, __half>(a);
    case 2: return launch_embed_out<Table::Dense, __nv_bfloat16>(a);
    default: return a.q4 ? launch_embed_out<Table::Q4, float>(a) : launch_embed_out<Table::Q5, float>(a);
  }
}

// order, sorted [n], count, parts [chunks][2][k], each on 256 bytes
size_t embed_backward_bytes(int64_t n, int k) {
  const int64_t c = chunk_of(n), chunks = (n + c - 1) / c;
  const size_t list = (static_cast<size_t>(n) * 4 + 255) / 256 * 256;
  return 256 + 2 * list + static_cast<size_t>(chunks) * 2 * k * sizeof(float);
}

cudaError_t launch_embed_backward(EmbedBackwardArgs a, void *workspace) {
  const size_t list = (static_cast<size_t>(a.n) * 4 + 255) / 256 * 256;
  uint8_t *w = static_cast<uint8_t *>(workspace);
  a.count = reinterpret_cast<int *>(w);
  a.order = reinterpret_cast<int *>(w + 256);
  a.sorted = reinterpret_cast<int *>(w + 256 + list);
  a.part = reinterpret_cast<float *>(w + 256 + 2 * list);
  a.chunk = static_cast<int>(chunk_of(a.n));
  if (a.out_dtype == 0) return launch_embed_backward_t<float>(a);
  if (a.out_dtype == 1) return launch_embed_backward_t<__half>(a);
  return launch_embed_backward_t<__nv_bfloat16>(a);
}

}  // namespace muse
