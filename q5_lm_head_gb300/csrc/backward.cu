// Backward pass of the output stage: the gradient by the logits back through
// soft cap, scale, the quantised matrix and the final norm.
//
// Per batch row b, with gl = dloss/dlogits and the forward's logits l:
//     t_v  = gl_v * scale * (cap > 0 ? (cap - l_v)(cap + l_v) / cap^2 : 1)
//     gx_k = sum_v t_v W_vk,     W_vk = d sc q - dmin m
// (t_v = 0 where l_v is outside -cap..cap: a masked logit, -infinity or a lowest
// value, did not come through the cap)
// and with the norm, r = 1/sqrt(mean h^2 + eps), xh = h r, gg = gx gamma:
//     gh = r (gg - xh mean(gg xh)),   ggamma = sum_b gx xh
//
// Bound: the CUDA cores' work between HBM and the tensor cores, no pipe of theirs
// alone: the full Q5_K head takes 215 us for one row, 402 us for 32, the Q4_K head
// 193 us for 8, 1.6, 2.8 and 1.7 times the time that HBM needs to read the matrix
// once.  For one row the main kernel issues in 73 % of all cycles and its integer
// pipe is busy in 67 % (Q4_K: 73 and 56 %: fewer operations a quant do not make it
// as much faster); the rest is roles that wait for one another.  For 32 rows it
// issues in 65 %: there the operand warps' work is nearly half the unpacking's and
// the products have four times the columns.  9 of 152 SMs have no CTA.
// The contraction runs along the rows v of W, across the direction in
// which its blocks are packed, so the tensor cores' A operand is W transposed: a
// lane of tensor memory is an input k, a column a pair of rows.
//
// Launches:
// 1. slope_kernel: t of every row, eight consecutive v of a batch row together,
//    and the largest of them (without the scale) of parts of each row, behind the
//    cap's slope: a label's gradient that a saturated logit lets nothing of through
//    would cost the others their low bits.  From it comes a power of two that brings a
//    row's t into f16's range.
// 2. backward_tc_kernel: a CTA takes two block columns (512 inputs) and a share
//    of the rows, 96 or 64 rows a stage.
//    * weight producer warp: a 2-D TMA box of the stage's rows x two blocks, in a
//      ring of its own: a slot is free again when it is unpacked, while the
//      operands wait for their products (one ring of both: 240 and 460 us).
//    * operand warps: read the blocks' d, dmin and scales.  With d = md 2^e,
//      1 <= |md| < 2, the power of two goes to the A side (A = sc (q - middle) 2^e,
//      at most 11 significant bits: exact in f16) and md, exact in f16 too, to the
//      B side: B = t md as the f16 pair (hi, lo), hi + lo = t md to 2^-21.  The
//      mins are a product of their own, A' = m 2^e' for the 16 sub-blocks,
//      B' = -t mdmin, with middle sc 2^e times B added to the same sums.
//    * four unpack warpgroups, two for each block, alternating between units of
//      16 to 48 rows: ldmatrix with transposition gives a thread four rows of
//      one input, and tcgen05.st (16 lanes x 128 bits) takes that fragment, the
//      rows in slab_order.
//    * MMA warp: per 16 rows four products of M = 128 (two nibble halves of two
//      blocks) and four small ones for mins and middles.  The tensor cores round
//      their sums towards zero, about 2^-24 a step, which over a share's thousand
//      steps would cost 1e-4 of the result: every 256 or 288 rows the unpack warps
//      add the accumulators to f32 sums of their own (5e-7).
//    The shares' sums go to the workspace.
// 3. finish_kernel: a cluster of CTAs a batch row adds the shares in their
//    order, undoes the power of two and does the norm's backward.
// 4. gamma_kernel (more than one batch row, gamma's gradient wanted).
//
// A block with |d| or |dmin| of 4 and more (weights in the thousands) would take
// B out of f16's range: the operand warps then set a flag and finish_kernel sums
// in f32 from the blocks themselves.
#include <atomic>
#include <cmath>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace muse {
namespace {

// Of the rows' largest |t|, all rows together, and so slope_kernel's CTAs: five an
// SM, all at once (32 rows 401 us; eight an SM, in two rounds, 404).
constexpr int kMaxParts = 760;
constexpr int kPadRows = 192;                 // t is kept, as zeros, up to a multiple of this
constexpr int kTileCols = 2 * kBlockWeights;  // inputs of a CTA
constexpr int kFlushRows = 256;               // between additions of the accumulators to the f32 sums, about
constexpr int kUnpackWarps = 16;
constexpr uint32_t kTmem = 512;

// ---------------------------------------------------------------- operands' scale
// What one of these kernels writes for the next is read through L2 (ld.cg): a
// kernel may have started while the one before it was still writing, and the
// read-only path is for data that no longer change.
//
// t is kept without the scale.  t 2^-e times the scale's mantissa in [2^11, 2^12) is
// below 2^13, with e = exponent of the row's largest |t| (0 for a row of zeros).
// Below 2^-115 it stays there, or the factor would leave f32's range: the operands
// then end at 2^-150 at least.
__device__ __forceinline__ int row_exponent(const float *gmax, int b, int parts) {
  float m = 0.0f;
  for (int i = threadIdx.x & 31; i < parts; i += 32) m = fmaxf(m, __ldcg(gmax + b * parts + i));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
  return m == 0.0f ? 0 : e < -115 ? -115 : e;   // 128 for infinities: they stay what they are
}
// A slab's 16 rows v in the order in which a thread's transposed fragment goes to
// tensor memory: the first two of every four, then the others.
__device__ __forceinline__ int slab_order(int v) { return (v & ~15) | ((v & 2) << 2) | ((v >> 1) & 6) | (v & 1); }

__device__ __forceinline__ float pow2(int e) {   // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// A masked logit, through which nothing goes back, whatever its gradient holds (a NaN is none).
__device__ __forceinline__ bool beyond_cap(float l, float cap) { return fabsf(l) > cap; }
// Each factor divided by itself: caps of 1e20 and more, whose square overflows, too.
__device__ __forceinline__ float cap_slope(float l, float cap, float inv_cap) {
  return ((cap - l) * inv_cap) * ((cap + l) * inv_cap);
}

// t[p/8][b][p%8] = gl * slope of row v, p = slab_order(v).
__global__ void __launch_bounds__(256) slope_kernel(const BackwardArgs a, int64_t share) {
  __shared__ float s_max[8];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the main kernel's set-up beside this one
  const int b = blockIdx.y;
  const int64_t row = static_cast<int64_t>(b) * a.n_rows;
  const float *g = a.grad_logits + row, *l = a.logits + row;
  const bool aligned = (row & 3) == 0;
  const int64_t fours = (a.n_rows + kPadRows - 1) / kPadRows * (kPadRows / 4);
  const int64_t lo = share * blockIdx.x, hi = lo + share < fours ? lo + share : fours;
  const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
  float m = 0.0f;
#pragma unroll 4
  for (int64_t i = lo + threadIdx.x; i < hi; i += 256) {
    const int64_t v = 4 * i;
    float x[4] = {}, y[4] = {};
    if (aligned && v + 4 <= a.n_rows) {
      const float4 t = __ldcs(reinterpret_cast<const float4 *>(g + v));
      x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
      if (a.cap > 0.0f) {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(l + v));
        y[0] = u.x, y[1] = u.y, y[2] = u.z, y[3] = u.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v + j < a.n_rows) {
          x[j] = __ldcs(g + v + j);
          if (a.cap > 0.0f) y[j] = __ldcs(l + v + j);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (a.cap > 0.0f && beyond_cap(y[j], a.cap)) x[j] = y[j] = 0.0f;
      if (a.cap > 0.0f) x[j] *= cap_slope(y[j], a.cap, inv_cap);
      m = fmaxf(m, fabsf(x[j]));
    }
    // slab_order: rows 4j, 4j + 1 to places 2j, 2j + 1 of the slab's first eight, the others to its second
    float *t = a.t + ((v >> 4 << 1) * a.batch + b) * 8 + ((v >> 1) & 6);
    *reinterpret_cast<float2 *>(t) = make_float2(x[0], x[1]);
    *reinterpret_cast<float2 *>(t + 8 * a.batch) = make_float2(x[2], x[3]);
  }
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) m = fmaxf(m, s_max[i]);
    a.gmax[b * gridDim.x + blockIdx.x] = m;
    if (blockIdx.x == 0 && b == 0) *a.flag = 0u;
  }
}

// ---------------------------------------------------------------- main kernel
template <int NM, bool kQ4>
struct BwdCfg {
  static constexpr int kBB = kQ4 ? kBlockBytesQ4 : kBlockBytes;
  // A box row is two blocks and the next 16 bytes: rows 368 (304) bytes apart put
  // eight rows' 16-byte pieces, which a transposing load takes at once, on all banks.
  static constexpr int kRowBytes = 2 * kBB + 16;
  // Rows of a stage: the more, the less the barriers of a stage cost (one row 223
  // us with units of 48 of them, 247 us with 64 rows in units of 32; 16 rows 286 and
  // 297 us); with 32 slots the stage's B tiles leave room for 64 (96 rows and two
  // operand slots: 498 us, against 402).
  static constexpr int kRows = NM <= 16 ? 96 : 64;
  static constexpr int kWBytes = kRows * kRowBytes;
  static constexpr int kN = 2 * NM;                               // B rows: hi, lo
  // Accumulator columns: with 8 slots hi and lo side by side (an MMA has 16
  // columns at least), else both into the same ones.
  static constexpr int kD = NM == 8 ? 16 : NM;
  // B: core matrices of 8 rows x 8 values; the rows are hi and lo of d and dmin
  // of both blocks (kinds 0-3), ordered so that one MMA's rows lie together: hi
  // and lo of a kind with 8 slots, else the kinds' hi, then their lo.  Core
  // matrices along v lie 16 bytes further apart than the rows are long: a warp's
  // stores fall on all banks.
  static constexpr int kBRows = 4 * kN;
  static constexpr int kLbo = kBRows * 16 + 16;
  static constexpr int kB = kRows / 8 * kLbo;                     // f16 [kBRows][kRows]
  __host__ __device__ static constexpr int row(int kind, int part) {
    return NM == 8 ? kind * 16 + part * 8 : part * 4 * NM + kind * NM;
  }
  static constexpr int kScl = 16 * kRows * 2;                     // f16 [2 blocks x 8][kRows]
  static constexpr int kSide = (kB + 2 * kScl + 127) / 128 * 128; // B; scales; mins
  static constexpr int kGroups = 2;                               // of four operand warps, taking the stages in turn
  static constexpr int kThreads = 32 * (kUnpackWarps + 4 * kGroups + 4);   // the weights' warp, two without a role, the MMAs'
  static constexpr int kT = 2 * 4 * kRows * 2;                    // a group's mantissas, f16, two stages of [4][kRows]
  // The mins' f32 sums (eight batch rows a warp): in shared memory (16 rows 276 us,
  // 283 in registers; eight of Q4_K 194 and 196); with 32 slots in registers until
  // the end, for their 2 KB would cost a slot of the weights' ring (404 and 402).
  static constexpr bool kMinsShared = NM <= 16;
  static constexpr int kMins = kMinsShared ? 16 * NM * 4 : 0;
  static_assert(kMinsShared || kGroups * kT >= 16 * NM * 4, "the mantissas' place at the end");
  static constexpr int kFixed = kGroups * kT + kMins + 512;       // and the barriers
  // Two rings: weights are free again as soon as they are unpacked, their
  // operands only when their products are done.  Of these three, or four with
  // 32 slots and fewer weights (414 us against 409), or two (one row 249 us
  // against 223).
  static constexpr int kSides = 3;
  static constexpr int kFit = (227 * 1024 - kFixed - kSides * kSide) / kWBytes;
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static_assert(kStages >= kSides && kWBytes % 128 == 0, "rings; the operand warps' waits count on the first");
  static constexpr int kSideAt = kStages * kWBytes, kMdAt = kSideAt + kSides * kSide;
  static constexpr int kSmem = kMdAt + kFixed;
  // Tensor memory: sets of sums of four M-tiles and two min products, then a ring
  // of units of kUS x 16 rows.  Two sets, so that one is added up while the other
  // is in use; with 32 slots one, or the ring would have two units of 16 rows only
  // (491 us for a full head of 32 rows, against 408).
  static constexpr int kSets = NM == 32 ? 1 : 2;
  static constexpr int kUS = NM <= 16 ? 3 : 2;
  static constexpr int kUnits = kRows / (16 * kUS);               // units a stage
  static constexpr int kSlab = 48;                                // columns of 16 rows: four M-tiles of 8, mins 8, scales 8
  static constexpr int kABase = kSets * 6 * kD;
  static constexpr int kBufs = (512 - kABase) / (kSlab * kUS);
  static_assert(kBufs >= 2 && kUnits == 2, "unit ring");
  static constexpr int kFlush = (kFlushRows + kRows - 1) / kRows;               // stages between flushes
  static constexpr uint32_t kIdesc = tc::idesc_f16_f32(128, kD), kIdescPair = tc::idesc_f16_f32(128, 2 * kD);
};

// 16 lanes x 8 columns: a and c lane t/4, b and d lane t/4 + 8, a and b column
// t%4, c and d column 4 + t%4.  (16x256b would take the rows in their order, at
// half the rate: 16 cycles for 32 lanes x 8 columns against 8.)
template <uint32_t kOffset>
__device__ __forceinline__ void st_16x128b(uint32_t ta, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0 + %5], {%1, %2, %3, %4};" ::"r"(ta), "r"(a), "r"(b), "r"(c),
               "r"(d), "n"(kOffset)
               : "memory");
}

// Two 16 x 16 byte matrices (rows at the addresses of lanes 0-15 and 16-31),
// transposed: lane t gets, in order, bytes t/4, t/4 + 8 of the first matrix's
// rows 4 (t%4) .. +3, and of the second's.
__device__ __forceinline__ void load_transposed(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kNeg1024 = 0xE400E400u;   // f16 pair (-1024, -1024)

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void tma_box(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(ptx::smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(ptx::smem_u32(bar)), "l"(policy)
      : "memory");
}

// Quants are taken out of a byte as 2^kLow q (low nibbles) and 2^kHigh q (high
// ones), their scales divided by as much.  In A stands (q - middle) sc, middle =
// 16 (Q5_K) or 8 (Q4_K): t sums to about 0 over a row, but its few large negative
// and many small positive values do so apart, and around the quants' middle
// neither part runs far ahead of the result (sums from 0 on had four times the
// rounding).  With the multiples, 1024 + 2^k middle has five significant bits and
// its product with a 6-bit scale is exact in f16, so one fma makes A.
template <bool kQ4>
struct Quant {
  static constexpr int kLow = kQ4 ? 3 : 2, kHigh = kQ4 ? 4 : 3;
  static constexpr float kMiddle = kQ4 ? 8.0f : 16.0f;
  static constexpr uint32_t kNegLow = kQ4 ? 0xE440E440u : 0xE440E440u;    // -(1024 + 64): 8 x 8, 4 x 16
  static constexpr uint32_t kNegHigh = kQ4 ? 0xE480E480u : 0xE480E480u;   // -(1024 + 128): 16 x 8, 8 x 16
};

// d (an f16 value) as md 2^e with -20 <= e <= 0 (a scale, and a sixteenth of it,
// is then exact in f16): 1 <= |md| < 2 apart from smaller values of d, up to 4
// where d is from 2 to 4; *big for more.
__device__ __forceinline__ float split_d(float d, int &e, bool &big) {
  const uint32_t bits = __float_as_uint(d);
  const int ex = static_cast<int>((bits >> 23) & 255) - 127;      // of the f16 value: -24 .. 15, -127 for 0
  big |= ex > 1;                                                  // infinities and NaN too
  e = ex > 0 ? 0 : ex < -20 ? -20 : ex;
  return d * pow2(-e);
}

template <int NM, bool kQ4>
__global__ void __launch_bounds__(BwdCfg<NM, kQ4>::kThreads, 1)
    backward_tc_kernel(const __grid_constant__ CUtensorMap wmap, const BackwardArgs a, float scale_m, int gparts, int pairs,
                       int splits) {
  using C = BwdCfg<NM, kQ4>;
  extern __shared__ __align__(1024) uint8_t smem[];                // [kStages][weights], [kSides][B tiles, scales, mins]
  __half *s_md = reinterpret_cast<__half *>(smem + C::kMdAt);      // [kGroups][kT]
  // [16 sub-blocks][NM]; in the mantissas' place once every stage's have been read, if not all along
  float *s_min = reinterpret_cast<float *>(smem + C::kMdAt + (C::kMinsShared ? C::kGroups * C::kT : 0));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kMdAt + C::kGroups * C::kT + C::kMins);
  uint64_t *wfull = bars, *wempty = wfull + C::kStages, *pfull = wempty + C::kStages, *pempty = pfull + C::kSides;
  uint64_t *tfull = pempty + C::kSides, *tempty = tfull + C::kBufs;
  uint64_t *dfull = tempty + C::kBufs, *dfree = dfull + 2, *done = dfree + 2;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(done + 1);
  volatile uint32_t *s_abort = s_tmem + 1;
  float *s_e2 = reinterpret_cast<float *>(s_tmem + 2);            // [NM] the scale's mantissa, rows of t into f16's range
  static_assert((2 * C::kStages + 2 * C::kSides + 2 * C::kBufs + 5) * 8 + 8 + 4 * NM <= 512, "behind the mantissas");

  // the warp's index from one lane: the compiler then knows the roles' branches and loops to be uniform
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int pair = blockIdx.x % pairs, split = blockIdx.x / pairs;   // neighbours stream the same rows
  const int64_t stages = (a.n_rows + C::kRows - 1) / C::kRows;
  const int64_t st0 = stages * split / splits;
  const int n_st = static_cast<int>(stages * (split + 1) / splits - st0);
  constexpr int kPrepThreads = 128;                               // of a group
  // The SM's scheduler of a warp is its index mod 4: the MMAs' goes to the one
  // whose unpack warps have no mins to store, the weights' to another.
  constexpr int kTmaWarp = kUnpackWarps + 4 * C::kGroups, kMmaWarp = kTmaWarp + 3;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(&wfull[i], 1);
      ptx::mbar_init(&wempty[i], kUnpackWarps);                   // the operand warps have read them before
    }
    for (int i = 0; i < C::kSides; ++i) {
      ptx::mbar_init(&pfull[i], 4);
      ptx::mbar_init(&pempty[i], 1);                              // the MMAs, which the unpack warps' reads come before
    }
    for (int i = 0; i < C::kBufs; ++i) {
      ptx::mbar_init(&tfull[i], kUnpackWarps / 2);
      ptx::mbar_init(&tempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&dfull[i], 1);
      ptx::mbar_init(&dfree[i], kUnpackWarps);
    }
    ptx::mbar_init(done, 1);
    *s_abort = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::alloc(s_tmem, kTmem);
    tc::relinquish();
  }
  if constexpr (C::kMinsShared)
    for (int i = tid; i < 16 * NM; i += C::kThreads) s_min[i] = 0.0f;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  constexpr uint32_t tbase = 0;                                   // the only allocation an SM has room for
  auto fail = [&]() {
    atomicOr(a.status, kStatusWaitTimeout);
    *s_abort = 1u;
  };
  // Bounded; gives up early once another role has.
  auto wait_one = [&](uint64_t *bar, uint32_t parity) {
    if (ptx::mbar_try_wait_nohint(bar, parity)) return true;
    for (uint32_t i = 0; i < ptx::kSpinLimit; ++i) {
      if (ptx::mbar_try_wait(bar, parity)) return true;
      if (*s_abort) return false;
    }
    return false;
  };
  auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_one(bar, parity)) != 0; };

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ weights
    asm volatile("griddepcontrol.wait;" ::: "memory");   // whatever wrote the weights is complete
    if (lane == 0) {
      const uint64_t policy = ptx::policy_evict_first();
      int issued = 0, slot = 0;
      uint32_t ph = 0;
      for (int i = 0; i < n_st; ++i) {
        if (i >= C::kStages && !wait_one(&wempty[slot], ph ^ 1u)) { fail(); break; }
        ptx::mbar_arrive_expect_tx(&wfull[slot], C::kWBytes);
        tma_box(smem + slot * C::kWBytes, &wmap, pair * (C::kBB / 2), static_cast<int>((st0 + i) * C::kRows), &wfull[slot],
                policy);
        issued = i + 1;
        if (++slot == C::kStages) { slot = 0; ph ^= 1u; }
      }
      // never leave copies in flight
      for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
        ptx::mbar_wait(&wfull[i % C::kStages], static_cast<uint32_t>((i / C::kStages) & 1));
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    // Tensor memory is addressed from 0 (all of it is this CTA's), descriptors
    // are a slot's first one plus a constant.  An MMA takes about 30 cycles here
    // (9 by itself with N = 16): it shares tensor memory with the unpack warps.
    const bool issuer = tc::elect_one();
    const uint64_t desc0 = tc::smem_desc_kmajor(ptx::smem_u32(smem + C::kSideAt), C::kLbo, 128);
    bool ok = true;
    int slot = 0, buf = 0;
    uint32_t pph = 0, tph = 0;
    for (int i = 0; i < n_st && ok; ++i) {
      const int period = i / C::kFlush, db = period % C::kSets;
      const bool opens = i % C::kFlush == 0;
      if (opens && period >= C::kSets && !(ok = wait(&dfree[db], ((period / C::kSets) & 1) ^ 1))) break;
      if (!(ok = wait(&pfull[slot], pph))) break;
      const uint64_t desc = desc0 + static_cast<uint64_t>(slot) * (C::kSide >> 4);
      const uint32_t d = db * 6 * C::kD;
#pragma unroll
      for (int u = 0; u < C::kUnits; ++u) {
        if (!(ok = wait(&tfull[buf], tph))) break;
        tc::fence_after();
        if (issuer) {
          const uint32_t ta = C::kABase + buf * (C::kUS * C::kSlab);
#pragma unroll
          for (int s = 0; s < C::kUS; ++s) {
            const bool acc = u > 0 || s > 0 || !opens;
#pragma unroll
            for (int part = 0; part < (NM == 8 ? 1 : 2); ++part) {
              // rows of B from (kind, part), 16 rows v from slab u * kUS + s
              auto b_at = [&](int kind) {
                return desc + ((C::row(kind, part) / 8 * 128 + (u * C::kUS + s) * 2 * C::kLbo) >> 4);
              };
#pragma unroll
              for (int mt = 0; mt < 4; ++mt)
                tc::mma_f16_tmemA(d + mt * C::kD, ta + s * C::kSlab + mt * 8, b_at(mt >> 1), C::kIdesc, acc || part > 0);
              // mins of both blocks by B', scales by B: a block's own columns are read, the other's are not
              tc::mma_f16_tmemA(d + 4 * C::kD, ta + s * C::kSlab + 32, b_at(2), C::kIdescPair, acc || part > 0);
              tc::mma_f16_tmemA(d + 4 * C::kD, ta + s * C::kSlab + 40, b_at(0), C::kIdescPair, true);
            }
          }
          tc::commit(&tempty[buf]);
        }
        __syncwarp();
        if (++buf == C::kBufs) { buf = 0; tph ^= 1u; }
      }
      if (!ok) break;
      if (issuer) {
        tc::commit(&pempty[slot]);
        if ((i + 1) % C::kFlush == 0 || i + 1 == n_st) tc::commit(&dfull[db]);
      }
      __syncwarp();
      if (++slot == C::kSides) { slot = 0; pph ^= 1u; }
    }
    if (!ok && lane == 0) fail();
    // tensor memory is freed only after every MMA issued here completed
    if (issuer) tc::commit(done);
    __syncwarp();
    if (!wait(done, 0) && lane == 0) fail();
  } else if (warp >= kUnpackWarps && warp < kTmaWarp) {
    // ------------------------------------------------------------ operands
    const int grp = (warp - kUnpackWarps) >> 2;                   // takes the stages grp, grp + kGroups, ..
    const int pt = tid - 32 * kUnpackWarps - kPrepThreads * grp;
    // this thread's tasks of a stage: eight rows v of one batch row
    constexpr int kOcts = C::kRows / 8, kStepB = kPrepThreads / kOcts, kTasks = (NM + kStepB - 1) / kStepB;
    // The schedulers' shares (a warp's is its index mod 4; 0 and 1 also have the
    // mins' stores, 3 the MMAs): a stage's headers beyond one a thread go to warps 0
    // and 2, B's tasks to warps 1, 3, 2, 0 in this order (one row of the full head 219
    // us, eight of Q4_K 206 then; headers by 0 and 1, B by 3, 2, 1, 0: 230 and 212).
    const int b_turn = 32 * (0x1203 >> (4 * (pt >> 5)) & 3) + lane;
    constexpr int kPasses = 2 * C::kRows > kPrepThreads ? 2 : 1;  // of the headers
    static_assert(2 * C::kRows <= kPrepThreads + 64, "the second by two warps");
    const int second = (pt & 32) == 0 ? kPrepThreads + (pt >> 6) * 32 + lane : 2 * C::kRows;
    const int oct = b_turn % kOcts, b_first = b_turn < kStepB * kOcts ? b_turn / kOcts : NM;
    asm volatile("griddepcontrol.wait;" ::: "memory");            // t and the rows' largest values
    for (int b = warp - kUnpackWarps; b < a.batch; b += 4 * C::kGroups) {
      const int e = row_exponent(a.gmax, b, gparts);
      if (lane == 0) s_e2[b] = scale_m * pow2(-(e >> 1)) * pow2((e >> 1) - e);   // in two: e is up to 128
    }
    float e2[kTasks];
    float4 t_next[kTasks][2];
    const float4 *t_at = reinterpret_cast<const float4 *>(a.t) + ((st0 + grp) * kOcts + oct) * a.batch * 2 + 2 * b_first;
    auto fetch = [&](bool any) {
#pragma unroll
      for (int j = 0; j < kTasks; ++j)
        if (any && b_first + j * kStepB < a.batch) {
          t_next[j][0] = __ldcg(t_at + 2 * j * kStepB);
          t_next[j][1] = __ldcg(t_at + 2 * j * kStepB + 1);
        }
      t_at += static_cast<int64_t>(C::kGroups) * kOcts * a.batch * 2;
    };
    fetch(grp < n_st);
    ptx::named_bar_sync(2 + C::kGroups, kPrepThreads * C::kGroups);
#pragma unroll
    for (int j = 0; j < kTasks; ++j) {
      const int b = b_first + j * kStepB;
      e2[j] = b < a.batch ? s_e2[b] : 0.0f;
    }
    bool bad = false, big = false;
    int turn = 0;
    for (int i = grp; i < n_st; i += C::kGroups, turn ^= 1) {
      const int slot = i % C::kStages, side_slot = i % C::kSides;
      __half *md_at = s_md + grp * (C::kT / 2) + turn * 4 * C::kRows;
      // The operands' slot first: stage i - kSides' products are done, so the box that was
      // in this weight slot before (stage i - kStages, an earlier one or the same) has landed,
      // and the parity means this stage's box.  With three weight slots that stage was the
      // other group's, whose boxes may land later than this one's.
      bad = (i >= C::kSides && !wait(&pempty[side_slot], ((i / C::kSides) & 1) ^ 1)) ||
            !wait(&wfull[slot], (i / C::kStages) & 1);
      const uint8_t *st = smem + slot * C::kWBytes;
      uint8_t *side = smem + C::kSideAt + side_slot * C::kSide;
      if (!bad) {
        // a block's header: powers of two with its scales and mins, mantissas for B
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass) {
          const int task = pass == 0 ? pt : second;
          if (task >= 2 * C::kRows) break;
          const int blk = task / C::kRows, row = task % C::kRows;
          const uint4 hdr = *reinterpret_cast<const uint4 *>(st + row * C::kRowBytes + blk * C::kBB);
          const float2 dd = __half22float2(*reinterpret_cast<const __half2 *>(&hdr.x));
          int ed, em;
          md_at[blk * C::kRows + slab_order(row)] = __float2half_rn(split_d(dd.x, ed, big));
          md_at[(2 + blk) * C::kRows + slab_order(row)] = __float2half_rn(-split_d(dd.y, em, big));
          // the quants come multiplied
          const uint32_t pd = pack_half2(pow2(ed - Quant<kQ4>::kLow), pow2(ed - Quant<kQ4>::kHigh));
          const uint32_t pm = pack_half2(pow2(em), pow2(em));
          const uint32_t sc[2] = {hdr.y & 0x3F3F3F3Fu, (hdr.w & 0x0F0F0F0Fu) | ((hdr.y >> 2) & 0x30303030u)};
          const uint32_t mn[2] = {hdr.z & 0x3F3F3F3Fu, ((hdr.w >> 4) & 0x0F0F0F0Fu) | ((hdr.z >> 2) & 0x30303030u)};
          __half *scl = reinterpret_cast<__half *>(side + C::kB) + blk * 8 * C::kRows + row;
          __half *mns = scl + 16 * C::kRows;
          const uint32_t one = 0x3C003C00u;
#pragma unroll
          for (int h = 0; h < 4; ++h) {                           // sub-blocks 2h, 2h + 1
            const uint32_t sel = h & 1 ? 0x4342u : 0x4140u;
            const uint32_t s = hmul2(hfma2(__byte_perm(sc[h >> 1], 0x64u, sel), one, kNeg1024), pd);
            const uint32_t m = hmul2(hfma2(__byte_perm(mn[h >> 1], 0x64u, sel), one, kNeg1024), pm);
            scl[(2 * h) * C::kRows] = __ushort_as_half(static_cast<unsigned short>(s));
            scl[(2 * h + 1) * C::kRows] = __ushort_as_half(static_cast<unsigned short>(s >> 16));
            mns[(2 * h) * C::kRows] = __ushort_as_half(static_cast<unsigned short>(m));
            mns[(2 * h + 1) * C::kRows] = __ushort_as_half(static_cast<unsigned short>(m >> 16));
          }
        }
      }
      if (ptx::named_bar_red_or(1 + grp, kPrepThreads, bad)) {
        bad = true;
        break;
      }
      // B tiles: the eight rows as hi and lo, for d and dmin of both blocks; the
      // columns of batch rows that are not there stay what they are, nobody reads their sums
#pragma unroll
      for (int j = 0; j < kTasks; ++j) {
        const int b = b_first + j * kStepB;
        if (b < a.batch) {
          const float4 t0 = t_next[j][0], t1 = t_next[j][1];
          // t as th + tl, once for the four kinds
          const float t[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
          uint32_t th[4], tl[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float x0 = t[2 * p] * e2[j], x1 = t[2 * p + 1] * e2[j];
            th[p] = pack_half2(x0, x1);
            const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&th[p]));
            tl[p] = pack_half2(x0 - h.x, x1 - h.y);
          }
          uint8_t *tile = side + oct * C::kLbo + (b >> 3) * 128 + (b & 7) * 16;
#pragma unroll
          for (int kind = 0; kind < 4; ++kind) {
            const uint4 m = *reinterpret_cast<const uint4 *>(md_at + kind * C::kRows + 8 * oct);
            const uint32_t md[4] = {m.x, m.y, m.z, m.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {       // (th + tl) md: th md rounded, its remainder (exact) and tl md
              hi[p] = hmul2(th[p], md[p]);
              lo[p] = hfma2(tl[p], md[p], hfma2(th[p], md[p], hi[p] ^ 0x80008000u));
            }
            *reinterpret_cast<uint4 *>(tile + C::row(kind, 0) / 8 * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(tile + C::row(kind, 1) / 8 * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the tiles, to the tensor cores' reads
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&pfull[side_slot]);
      fetch(i + C::kGroups < n_st);
    }
    if (bad && lane == 0) fail();
    if (big) atomicOr(a.flag, 1u);
  } else if (warp < kUnpackWarps) {
    // ------------------------------------------------------------ unpacking
    const int blk = (warp >> 2) & 1, par = warp >> 3, wq = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t rot = static_cast<uint32_t>(6 - 2 * wq) & 31u;   // high bit 2wq -> 6, 2wq + 1 -> 7
    // what this warpgroup's small operand is multiplied by: 1 for mins, the middle
    // for scales (divided as sub-block lane/4's)
    const int k_divided = (lane >> 2) & 1 ? Quant<kQ4>::kHigh : Quant<kQ4>::kLow;
    const float middle1 = blk ? Quant<kQ4>::kMiddle * pow2(k_divided) : 1.0f;
    const uint32_t middle = pack_half2(middle1, middle1);
    const uint32_t src0 = ptx::smem_u32(smem) + (lane & 15) * C::kRowBytes + blk * C::kBB + 16 * (lane >> 4);
    // the f32 sums: inputs of M-tile warp/4 by batch row, and mins (lane: sub-block) of eight batch rows
    const int mt = warp >> 2;
    // mins: warpgroup mt's warp of quarter `mblk` reads block mblk's eight sub-blocks, batch rows 8 mt'..
    const int mblk = wq, mcol = NM == 8 ? 0 : 8 * mt;
    const bool min_warp = NM == 8 ? wq < 2 && mt == 2 * wq : wq < 2 && mt < NM / 8;
    unsigned long long sum[NM / 2];             // pairs of batch rows
    float msum[8] = {};                         // eight batch rows, if not in s_min
#pragma unroll
    for (int j = 0; j < NM / 2; ++j) sum[j] = 0ull;
    int flushed = 0;
    auto flush = [&]() {
      const int db = flushed % C::kSets;
      if (!wait(&dfull[db], (flushed / C::kSets) & 1)) return false;
      tc::fence_after();
      const uint32_t d = tbase + db * 6 * C::kD;
#pragma unroll
      for (int c0 = 0; c0 < C::kD; c0 += 16) {
        if (c0 == 0 || c0 < a.batch) {
          uint32_t x[16];
          tc::ld_32x32b_x16(d + lane_base + mt * C::kD + c0, x);
          tc::wait_ld();
          auto two = [&](int j) { return pack2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])); };
          if constexpr (NM == 8) {              // hi and lo
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (2 * j < a.batch) sum[j] = add2(sum[j], add2(two(2 * j), two(8 + 2 * j)));
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[c0 / 2 + j] = add2(sum[c0 / 2 + j], two(2 * j));
          }
        }
      }
      if (min_warp) {
#pragma unroll
        for (int h = 0; h < (NM == 8 ? 2 : 1); ++h) {
          uint32_t x[8];
          tc::ld_32x32b_x8(d + lane_base + (4 + mblk) * C::kD + mcol + 8 * h, x);
          tc::wait_ld();
          if constexpr (!C::kMinsShared) {
#pragma unroll
            for (int j = 0; j < 8; ++j) msum[j] += __uint_as_float(x[j]);
          } else if (lane < 8) {
            float4 *at = reinterpret_cast<float4 *>(s_min + (8 * mblk + lane) * NM + mcol);   // this warp's own
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float4 m = at[j];
              m.x += __uint_as_float(x[4 * j]);
              m.y += __uint_as_float(x[4 * j + 1]);
              m.z += __uint_as_float(x[4 * j + 2]);
              m.w += __uint_as_float(x[4 * j + 3]);
              at[j] = m;
            }
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&dfree[db]);
      ++flushed;
      return true;
    };
    bool ok = true;
    int slot = 0, side_slot = 0, buf = par, unit = par;   // unit: of the whole share; its buffer is unit % kBufs
    uint32_t pph = 0, tph = 0;
    for (int i = 0; i < n_st; ++i) {
      if (!(ok = wait(&pfull[side_slot], pph))) break;    // the weights too: the operand warps have waited for them
      const uint8_t *side = smem + C::kSideAt + side_slot * C::kSide;
      const __half *k_at = reinterpret_cast<const __half *>(side + C::kB) + 4 * (lane & 3);
      const __half *scl = k_at + (blk * 8 + 2 * wq) * C::kRows;
      // of sub-block lane/4 of block wq: the mins for one warpgroup, the scales for the other
      const __half *small = k_at + ((blk ? 0 : 16) + 8 * (wq & 1) + (lane >> 2)) * C::kRows;
      // One unit of a stage's two.  With two buffers the compiler is to know that, and
      // which buffer it is (one row 219 -> 215 us, eight of Q4_K 199 -> 194); with 32
      // slots what it then keeps in registers makes others spill (403 -> 416 us).
      for (int u = par; u < (C::kBufs == 2 ? par + 1 : C::kUnits); u += 2) {
        if ((C::kBufs == 2 || unit >= C::kBufs) && !(ok = wait(&tempty[buf], tph ^ 1u))) break;   // the first finds it free
        tc::fence_after();
        const uint32_t at0 = tbase + lane_base + C::kABase + buf * C::kUS * C::kSlab, at_small = at0 + 8 * blk;
        const uint32_t src1 = src0 + slot * C::kWBytes + u * C::kUS * 16 * C::kRowBytes;
        auto slab_to_tmem = [&](auto s_const) {
          constexpr int s = decltype(s_const)::value;
          const int slab = u * C::kUS + s;
          const uint32_t src = src1 + s * 16 * C::kRowBytes;
          uint32_t q[4], h[4];
          load_transposed(src + (kQ4 ? kOffQsQ4 : kOffQs) + 32 * wq, q);
          if constexpr (!kQ4) load_transposed(src + kOffQh, h);
          const uint2 k0 = *reinterpret_cast<const uint2 *>(scl + 16 * slab);              // low nibbles' scales
          const uint2 k1 = *reinterpret_cast<const uint2 *>(scl + C::kRows + 16 * slab);   // high ones', divided
          uint2 m = make_uint2(0u, 0u);
          if (wq < 2) m = *reinterpret_cast<const uint2 *>(small + 16 * slab);
          using Q = Quant<kQ4>;
          const uint32_t a00 = hmul2(k0.x, Q::kNegLow), a01 = hmul2(k0.y, Q::kNegLow);
          const uint32_t a10 = hmul2(k1.x, Q::kNegHigh), a11 = hmul2(k1.y, Q::kNegHigh);
          const uint32_t at = at0 + 16 * blk;
          uint32_t lo[8], hi[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            uint32_t ql, qh;
            if constexpr (kQ4) {
              ql = (q[r] << 3) & 0x78787878u;
              qh = q[r] & 0xF0F0F0F0u;
            } else {
              const uint32_t hr = __funnelshift_l(h[r], h[r], rot);
              ql = ((q[r] << 2) & 0x3C3C3C3Cu) | (hr & 0x40404040u);
              qh = ((q[r] >> 1) & 0x78787878u) | (hr & 0x80808080u);
            }
            lo[2 * r] = hfma2(__byte_perm(ql, 0x64u, 0x4140u), k0.x, a00);      // (1024 + 4q) s/4 - 1088 s/4, exact
            lo[2 * r + 1] = hfma2(__byte_perm(ql, 0x64u, 0x4342u), k0.y, a01);
            hi[2 * r] = hfma2(__byte_perm(qh, 0x64u, 0x4140u), k1.x, a10);
            hi[2 * r + 1] = hfma2(__byte_perm(qh, 0x64u, 0x4342u), k1.y, a11);
          }
          constexpr uint32_t kAt = s * C::kSlab, kUp = 16u << 16;
          st_16x128b<kAt>(at, lo[0], lo[2], lo[1], lo[3]);
          st_16x128b<kAt + kUp>(at, lo[4], lo[6], lo[5], lo[7]);
          st_16x128b<kAt + 8>(at, hi[0], hi[2], hi[1], hi[3]);
          st_16x128b<kAt + kUp + 8>(at, hi[4], hi[6], hi[5], hi[7]);
          // block wq's mins or scales times the middle: lanes 0-7 of this quarter (and, unread, 8-15)
          if (wq < 2) {
            m.x = hmul2(m.x, middle);
            m.y = hmul2(m.y, middle);
            st_16x128b<kAt + 32>(at_small, m.x, m.x, m.y, m.y);
          }
        };
        slab_to_tmem(std::integral_constant<int, 0>{});
        if constexpr (C::kUS > 1) slab_to_tmem(std::integral_constant<int, 1>{});
        if constexpr (C::kUS > 2) slab_to_tmem(std::integral_constant<int, 2>{});
        if constexpr (C::kUS > 3) slab_to_tmem(std::integral_constant<int, 3>{});
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&tfull[buf]);
        unit += 2;
        if constexpr (C::kBufs == 2) {
          tph ^= 1u;
        } else if ((buf += 2) >= C::kBufs) {
          buf -= C::kBufs;
          tph ^= 1u;
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&wempty[slot]);
      if (++slot == C::kStages) slot = 0;
      if (++side_slot == C::kSides) { side_slot = 0; pph ^= 1u; }
      // the set before the one now in use; or the only set, one stage after its last (the ring holds that stage)
      const bool due = C::kSets == 2 ? (i + 1) % C::kFlush == 0 && i + 1 > C::kFlush : i % C::kFlush == 0 && i > 0;
      if (due && !(ok = flush())) break;
    }
    while (ok && flushed < (n_st + C::kFlush - 1) / C::kFlush) ok = flush();
    if (!ok && lane == 0) fail();
    if constexpr (!C::kMinsShared)
      if (min_warp && ok && lane < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s_min[(8 * mblk + lane) * NM + mcol + j] = msum[j];
      }
    ptx::named_bar_sync(1 + C::kGroups, 32 * kUnpackWarps);
    const int kc = pair * kTileCols + (mt >> 1) * kBlockWeights + 64 * wq + 32 * (mt & 1) + lane;
    if (ok && kc < a.k) {
      const float *mins = s_min + ((mt >> 1) * 8 + 2 * wq + (mt & 1)) * NM;
      float *out = a.part + static_cast<int64_t>(split) * a.batch * a.k + kc;
#pragma unroll
      for (int b = 0; b < NM; b += 2) {
        const float2 x = unpack2(sum[b / 2]);
        if (b < a.batch) out[static_cast<int64_t>(b) * a.k] = x.x + mins[b];
        if (b + 1 < a.batch) out[static_cast<int64_t>(b + 1) * a.k] = x.y + mins[b + 1];
      }
    }
    tc::fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(*s_tmem, kTmem);
  }
}

// ---------------------------------------------------------------- shares' sum and norm
constexpr int kFinishThreads = 256;

// gx of batch row b at column j from the blocks themselves, in f32.
template <bool kQ4>
__device__ float plain_sum(const BackwardArgs &a, int b, int j) {
  constexpr int kBB = kQ4 ? kBlockBytesQ4 : kBlockBytes;
  constexpr int kQs = kQ4 ? kOffQsQ4 : kOffQs;
  const int kb = j / kBlockWeights, s = j % kBlockWeights / 32, l = j % 32;
  float sum = 0.0f;
  for (int64_t v0 = 0; v0 < a.n_rows; v0 += 512) {                // sums of 512, then of those: a short chain
    float part = 0.0f;
    for (int64_t v = v0; v < v0 + 512 && v < a.n_rows; ++v) {
      const int64_t at = static_cast<int64_t>(b) * a.n_rows + v;
      float t = a.grad_logits[at] * a.scale;
      if (a.cap > 0.0f) t = beyond_cap(a.logits[at], a.cap) ? 0.0f : t * cap_slope(a.logits[at], a.cap, 1.0f / a.cap);
      const uint8_t *blk = a.w + (v * (a.k / kBlockWeights) + kb) * kBB;
      const uint4 hdr = __ldg(reinterpret_cast<const uint4 *>(blk));
      const float2 dd = __half22float2(*reinterpret_cast<const __half2 *>(&hdr.x));
      int sc, mn;
      q5k_scale_min(hdr.y, hdr.z, hdr.w, s, sc, mn);
      int q = (blk[kQs + 32 * (s >> 1) + l] >> (4 * (s & 1))) & 15;
      if (!kQ4) q |= ((blk[kOffQh + l] >> s) & 1) << 4;
      part = fmaf(t, fmaf(dd.x * static_cast<float>(sc), static_cast<float>(q), -dd.y * static_cast<float>(mn)), part);
    }
    sum += part;
  }
  return sum;
}

__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const BackwardArgs a, int splits, int gparts, int scale_e) {
  __shared__ float s_red[2][kFinishThreads / 32];
  __shared__ float s_from[2][16];
  const int tid = threadIdx.x;
  const uint32_t cr = cluster_rank(), cs = cluster_size();
  const int b = blockIdx.x / cs;
  const int lo = static_cast<int>(static_cast<int64_t>(a.k / 4) * cr / cs) * 4;
  const int hi = static_cast<int>(static_cast<int64_t>(a.k / 4) * (cr + 1) / cs) * 4;
  cluster_arrive();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.grad_gamma && a.batch > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // gamma_kernel follows
  const bool plain = __ldcg(a.flag) != 0u;
  const double back = ldexp(1.0, row_exponent(a.gmax, b, gparts) + scale_e);
  const int64_t stride = static_cast<int64_t>(a.batch) * a.k;
  float *gx = a.part + static_cast<int64_t>(b) * a.k;
  const int64_t at = static_cast<int64_t>(b) * a.k;
  float ss = 0.0f, dot = 0.0f;
  for (int j = lo + 4 * tid; j < hi; j += 4 * kFinishThreads) {
    float x[4] = {};
    if (!plain) {
      float4 s = __ldcg(reinterpret_cast<const float4 *>(gx + j));
#pragma unroll 8
      for (int p = 1; p < splits; ++p) {
        const float4 o = __ldcg(reinterpret_cast<const float4 *>(gx + p * stride + j));
        s.x += o.x;
        s.y += o.y;
        s.z += o.z;
        s.w += o.w;
      }
      x[0] = static_cast<float>(s.x * back);
      x[1] = static_cast<float>(s.y * back);
      x[2] = static_cast<float>(s.z * back);
      x[3] = static_cast<float>(s.w * back);
    } else {
      for (int i = 0; i < 4; ++i) x[i] = a.q4 ? plain_sum<true>(a, b, j + i) : plain_sum<false>(a, b, j + i);
    }
    const float4 r = make_float4(x[0], x[1], x[2], x[3]);
    if (!a.gamma) {
      *reinterpret_cast<float4 *>(a.grad_hidden + at + j) = r;
    } else {
      *reinterpret_cast<float4 *>(gx + j) = r;                    // read again below, and for gamma
      const float4 h = *reinterpret_cast<const float4 *>(a.hidden + at + j);
      const float4 g = *reinterpret_cast<const float4 *>(a.gamma + j);
      ss = fmaf(h.x, h.x, fmaf(h.y, h.y, fmaf(h.z, h.z, fmaf(h.w, h.w, ss))));
      dot = fmaf(r.x * g.x, h.x, fmaf(r.y * g.y, h.y, fmaf(r.z * g.z, h.z, fmaf(r.w * g.w, h.w, dot))));
    }
  }
  cluster_wait();                         // every CTA of the cluster has started
  if (!a.gamma) return;
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    dot += __shfl_xor_sync(0xffffffffu, dot, o);
  }
  if ((tid & 31) == 0) {
    s_red[0][tid >> 5] = ss;
    s_red[1][tid >> 5] = dot;
  }
  __syncthreads();
  if (tid < static_cast<int>(cs)) {
    ss = dot = 0.0f;
    for (int i = 0; i < kFinishThreads / 32; ++i) {
      ss += s_red[0][i];
      dot += s_red[1][i];
    }
    peer_store32(peer_addr(&s_from[0][cr], tid), __float_as_uint(ss));
    peer_store32(peer_addr(&s_from[1][cr], tid), __float_as_uint(dot));
  }
  cluster_sync();
  ss = dot = 0.0f;
  for (uint32_t i = 0; i < cs; ++i) {
    ss += s_from[0][i];
    dot += s_from[1][i];
  }
  const float r = 1.0f / sqrtf(ss / static_cast<float>(a.k) + a.eps);
  const float c = r * r * dot / static_cast<float>(a.k);
  if (cr == 0 && tid == 0) a.rms[b] = r;
  for (int j = lo + 4 * tid; j < hi; j += 4 * kFinishThreads) {
    const float4 x = *reinterpret_cast<const float4 *>(gx + j);
    const float4 h = *reinterpret_cast<const float4 *>(a.hidden + at + j);
    const float4 g = *reinterpret_cast<const float4 *>(a.gamma + j);
    *reinterpret_cast<float4 *>(a.grad_hidden + at + j) = make_float4(
        r * (x.x * g.x - h.x * c), r * (x.y * g.y - h.y * c), r * (x.z * g.z - h.z * c), r * (x.w * g.w - h.w * c));
    if (a.grad_gamma && a.batch == 1)
      *reinterpret_cast<float4 *>(a.grad_gamma + j) = make_float4(x.x * h.x * r, x.y * h.y * r, x.z * h.z * r, x.w * h.w * r);
  }
}

__global__ void __launch_bounds__(128) gamma_kernel(const BackwardArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int j = blockIdx.x * 128 + threadIdx.x;
  float v = 0.0f;
#pragma unroll 8
  for (int b = 0; b < a.batch; ++b) {
    const int64_t at = static_cast<int64_t>(b) * a.k + j;
    v = fmaf(__ldcg(a.part + at) * __ldcg(a.rms + b), a.hidden[at], v);
  }
  a.grad_gamma[j] = v;
}

// ---------------------------------------------------------------- host side
int bwd_pairs(int k) { return (k / kBlockWeights + 1) / 2; }
// As many shares of the rows as leave each SM one CTA.
int bwd_splits(int64_t n_rows, int k, int num_sms, int rows) {
  const int64_t stages = (n_rows + rows - 1) / rows;
  int64_t s = num_sms / bwd_pairs(k);
  if (s < 1) s = 1;
  return static_cast<int>(s < stages ? s : stages);
}

// The matrix in boxes of `rows` rows x `bytes` bytes (a multiple of 16, as the
// blocks are: every box starts on a 16-byte boundary), beyond its edges zeros.
// Encoded anew by every call: nothing is kept by the weights' address.
cudaError_t encode_boxes(CUtensorMap *map, const BackwardArgs &a, int bytes, int rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 enc = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    cudaDriverEntryPointQueryResult q;
    void *p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return nullptr;
  }();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t row = static_cast<cuuint64_t>(a.k / kBlockWeights) * (a.q4 ? kBlockBytesQ4 : kBlockBytes);
  const cuuint64_t dims[2] = {row / 4, static_cast<cuuint64_t>(a.n_rows)};
  const cuuint64_t strides[1] = {row};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(bytes / 4), static_cast<cuuint32_t>(rows)};
  const cuuint32_t steps[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t *>(a.w), dims, strides, box, steps,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                             A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start before the previous grid ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...);
}

template <int NM, bool kQ4>
cudaError_t launch_backward_nm(const BackwardArgs &a, float scale_m, int gparts, int *splits) {
  using C = BwdCfg<NM, kQ4>;
  CUtensorMap map;
  cudaError_t e = encode_boxes(&map, a, C::kRowBytes, C::kRows);
  if (e != cudaSuccess) return e;
  static std::atomic<unsigned long long> configured{0};   // one bit per device; host threads may race here
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(backward_tc_kernel<NM, kQ4>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int pairs = bwd_pairs(a.k);
  *splits = bwd_splits(a.n_rows, a.k, a.num_sms, C::kRows);
  return launch_dependent(backward_tc_kernel<NM, kQ4>, dim3(static_cast<unsigned>(pairs * *splits)), C::kThreads, C::kSmem,
                          1, a.stream, map, a, scale_m, gparts, pairs, *splits);
}

}  // namespace

size_t backward_part_floats(int64_t n_rows, int k, int max_batch, int num_sms) {
  return static_cast<size_t>(bwd_splits(n_rows, k, num_sms, 64)) * max_batch * k;
}
size_t backward_t_floats(int64_t n_rows, int max_batch) {
  return static_cast<size_t>((n_rows + kPadRows - 1) / kPadRows * kPadRows) * max_batch;
}
size_t backward_misc_floats() { return kMaxParts + 32 + 1; }   // largest |t|, RMS factors, flag

cudaError_t launch_backward(const BackwardArgs &a) {
  // the scale as scale_m 2^scale_e, 2^11 <= |scale_m| < 2^12
  int scale_e = 0;
  const float scale_m = std::ldexp(std::frexp(a.scale, &scale_e), 12);
  scale_e -= 12;
  // rows of t in fours: one a thread at least, shares of whole CTAs
  const int64_t ctas = (a.n_rows + kPadRows - 1) / kPadRows * (kPadRows / 4) / 256 + 1, most = kMaxParts / a.batch;
  const int64_t share = (ctas + most - 1) / most * 256;
  const int gparts = static_cast<int>((ctas * 256 + share - 1) / share);
  // an ordinary launch: after everything before it on the stream, the weights' own writer too
  slope_kernel<<<dim3(static_cast<unsigned>(gparts), static_cast<unsigned>(a.batch)), 256, 0, a.stream>>>(a, share);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  int splits = 1;
  const int slots = tc_batch_slots(a.batch);
  if (a.q4)
    e = slots == 8    ? launch_backward_nm<8, true>(a, scale_m, gparts, &splits)
        : slots == 16 ? launch_backward_nm<16, true>(a, scale_m, gparts, &splits)
                      : launch_backward_nm<32, true>(a, scale_m, gparts, &splits);
  else
    e = slots == 8    ? launch_backward_nm<8, false>(a, scale_m, gparts, &splits)
        : slots == 16 ? launch_backward_nm<16, false>(a, scale_m, gparts, &splits)
                      : launch_backward_nm<32, false>(a, scale_m, gparts, &splits);
  if (e != cudaSuccess) return e;
  // eight CTAs a row, or one with little to add (5 rows of 2,048 x 6,656: 12.5 us as a
  // whole, against 22.7 us with one each; one row of the full head 224 us against 238)
  const int cs = a.k >= 2048 ? 8 : 1;
  e = launch_dependent(finish_kernel, dim3(static_cast<unsigned>(a.batch * cs)), kFinishThreads, 0, cs, a.stream, a, splits,
                       gparts, scale_e);
  if (e != cudaSuccess || !a.grad_gamma || a.batch == 1) return e;
  return launch_dependent(gamma_kernel, dim3(static_cast<unsigned>(a.k / 128)), 128, 0, 1, a.stream, a);
}

}  // namespace muse
