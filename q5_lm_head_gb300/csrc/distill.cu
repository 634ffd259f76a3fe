// Distillation from a teacher's top alternatives: each row's loss and its
// gradient by the student's logits.
//
// Student row x of V logits, z = x / T, q = softmax(z).  Teacher entries
// (id_j, l_j), those with an id outside 0..V-1 left out, S the set of ids:
//     renormalised: p_j = exp(l_j) / sum exp(l),  p_t = 0
//     tail:         p_j = exp(l_j),  p_t = max(0, 1 - sum p),  q_t = sum_{i not in S} q_i
//     loss = w [ sum_j p_j (log p_j - log q_{id_j}) + p_t (log p_t - log q_t) ]
//     dloss/dx_i = w/T [ (sum p + p_t) q_i - sum_{j: id_j = i} p_j - [i not in S] p_t q_i / q_t ]
//
// Bound: HBM, each logit read once and each gradient written once (1,024 bf16 rows
// of 202,048: 166 us, 5.0 TB/s, 73 % of the measured copy rate; the rest are the
// row's barriers, which the SM's other CTAs do not quite cover).  A cluster
// of CTAs holds a row in its shared memory (in the logits' type, up to 52 KB a
// CTA, so that four CTAs of an SM overlap their loads, sums and stores), and one
// barrier of the cluster joins the CTAs' maxima and sums.  The sum
// outside S is taken apart from the sum inside, not as a difference: where the
// student is sure of the teacher's ids a difference would be rounding alone.
// The ids' values are taken out of the row (set to -infinity) before the sum.
// Each of the two sums goes with a maximum of its own, m_r outside S and m_i inside,
// for the two may lie hundreds of binary orders apart: against the row's maximum the
// smaller would be 0 in 32 bits, its logarithm and its shares are ordinary numbers.
// So, with R = sum_{i not in S} 2^((x_i - m_r) c) >= 1 and Z the row's sum against m,
//     log q_t = (m_r - m)/T + log R - log Z
//     dloss/dx_i = 2^((x_i - m_r) c) w/T [ (sum p + p_t) 2^((m_r - m) c) / Z - p_t / R ],  i not in S:
// one factor for the whole row, which cannot overflow.
// Nothing is kept in global memory, so calls may overlap.  A row that 16 CTAs
// cannot hold is read by one CTA, twice for the loss and once more for the gradient.
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace muse {
namespace {

constexpr int kDistillThreads = 256;
constexpr int kDistillWarps = kDistillThreads / 32;
constexpr int kDistillCluster = 16;
constexpr int kHeldFour = 52 * 1024;     // bytes of a row in a CTA: four CTAs an SM
constexpr int kHeldOne = 216 * 1024;     // one CTA an SM

struct DistillShared {
  __align__(16) int id[kMaxTop];         // -1: left out
  float p[kMaxTop], lp[kMaxTop];         // probability and its logarithm
  float x[kMaxTop];                      // the ids' logits: this CTA's own; all of them in the first CTA
  float rest_m[kDistillWarps], rest[kDistillWarps], in_m[kDistillWarps], in[kDistillWarps];   // the warps' maxima and sums
  float mass;
  int twice[2];                          // an id of this half of the entries has come before
  float from_rest_m[kDistillCluster], from_rest[kDistillCluster], from_in_m[kDistillCluster], from_in[kDistillCluster];
};

__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

// Sums against the maximum m (m = -infinity: only 0, or NaN) onto another one.
__device__ __forceinline__ float move_sum(float s, float from, float to, float c) {
  return to == -INFINITY || s == 0.0f ? s : s * exp2_approx(shift_exponent(from, to, c));
}
__device__ __forceinline__ float warp_max(float v) {
  return order_key_float(__reduce_max_sync(0xffffffffu, float_order_key(v)));
}
// What the teacher's entries leave for the rest; a NaN among them stays one.
__device__ __forceinline__ float left_over(float mass) { return mass > 1.0f ? 0.0f : 1.0f - mass; }
// -infinity as a reference: 0, against which nothing but 0 or NaN is summed.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

template <typename T>
__global__ void __launch_bounds__(kDistillThreads, 4) distill_kernel(const DistillArgs a) {
  constexpr int W = Vec<T>::W;
  extern __shared__ __align__(16) uint8_t held[];
  __shared__ DistillShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t cr = cluster_rank(), cs = cluster_size();
  const int cs_log = 31 - __clz(cs);      // a power of two
  const int64_t row = blockIdx.x >> cs_log;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  T *g = a.grad ? static_cast<T *>(a.grad) + row * a.grad_ld : nullptr;
  const int v = static_cast<int>(a.v), k = a.n_top;
  const float c = a.exponent_scale;       // log2(e) / temperature
  const bool apart = a.tail;              // the sums inside and outside the ids are wanted one by one
  cluster_arrive();                       // waited for before the first store to a peer

  // this CTA's share: head values (first CTA), vectors [v0, v1), the rest (last CTA)
  const RowCut cut = cut_row(x, v);
  const int v0 = static_cast<int>((static_cast<int64_t>(cut.vecs) * cr) >> cs_log);
  const int v1 = static_cast<int>((static_cast<int64_t>(cut.vecs) * (cr + 1)) >> cs_log);
  const int first = cut.head + v0 * W;    // index of the first held value
  const int count = (v1 - v0) * W;
  T *row_held = reinterpret_cast<T *>(held);
  uint4 *vec_held = reinterpret_cast<uint4 *>(held);
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + cut.head) + v0;
  const int rest_n = v - cut.head - cut.vecs * W;
  int edge_i = -1;                        // a value beside the vectors, one thread's own
  if (cr == 0 && tid < cut.head) edge_i = tid;
  if (cr == cs - 1 && tid >= 32 && tid < 32 + rest_n) edge_i = v - rest_n + tid - 32;

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the logits and the teacher's side are complete
  const float w = a.row_weight ? a.row_weight[row] : 1.0f;
  float scale = w * a.inv_temperature, f_in = 0.0f, f_out = 0.0f;
  float edge = -INFINITY;
  bool edge_in = false;
  int own = -1;                           // the place of this thread's teacher entry in row_held
  bool again = false;                     // an earlier entry has the same id
  if (w != 0.0f) {
    for (int i = tid; i < v1 - v0; i += kDistillThreads) copy_async16(vec_held + i, xv + i);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (edge_i >= 0) edge = to_float(x[edge_i]);
    if (tid < kMaxTop) {
      const int id = tid < k ? a.teacher_ids[row * k + tid] : -1;
      const float l = tid < k ? a.teacher_logprobs[row * k + tid] : -INFINITY;
      const bool ok = id >= 0 && id < v;
      sh.id[tid] = ok ? id : -1;
      sh.lp[tid] = ok ? l : -INFINITY;
      if (id >= first && id < first + count) own = id - first;
      const uint32_t same = __match_any_sync(0xffffffffu, ok ? id : -1 - lane);
      again = __ffs(same) - 1 != lane;
      ptx::named_bar_sync(1, kMaxTop);
      if (warp == 1 && k > 32) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const int4 o = *reinterpret_cast<const int4 *>(sh.id + j);
          again |= ok && (o.x == id || o.y == id || o.z == id || o.w == id);
        }
      }
      const bool any = __any_sync(0xffffffffu, again);
      if (lane == 0) sh.twice[warp] = any;
    }
    if (warp == 0) {                      // the teacher's probabilities
      float l0 = sh.lp[lane], l1 = sh.lp[lane + 32];
      if (!a.tail) {
        float top = fmaxf(l0, l1);
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top > -INFINITY) {            // the differences first: teacher logits may be thousands in size
          l0 -= top;
          l1 -= top;
          float s = expf(l0) + expf(l1);
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          s = logf(s);
          l0 -= s;
          l1 -= s;
        }
      }
      const float p0 = expf(l0), p1 = expf(l1);
      float mass = p0 + p1;
      for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
      sh.lp[lane] = l0;
      sh.lp[lane + 32] = l1;
      sh.p[lane] = p0;
      sh.p[lane + 32] = p1;
      if (lane == 0) sh.mass = mass;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // the ids' values out of the row
    float mine = -INFINITY, in_m = -INFINITY;
    if (tid < kMaxTop) {
      if (own >= 0) in_m = mine = to_float(row_held[own]);
      ptx::named_bar_sync(1, kMaxTop);    // an id given twice: both have read it
      if (own >= 0) {
        row_held[own] = from_float<T>(-INFINITY);
        sh.x[tid] = mine;
      }
    }
    if (edge_i >= 0)
      for (int j = 0; j < k; ++j)
        if (sh.id[j] == edge_i) {
          edge_in = true;
          sh.x[j] = edge;
        }
    __syncthreads();

    // maximum and sum of what is left: two passes over shared memory, so that no
    // sum moves onto a new maximum on the way
    float top = -INFINITY;
    {
      uint4 most = vec_lowest(T{});
      for (int i = tid; i < v1 - v0; i += kDistillThreads) most = vec_max(most, vec_held[i], T{});
      float o[W];
      unpack(most, o, T{});
#pragma unroll
      for (int j = 0; j < W; ++j) top = fmaxf(top, o[j]);
    }
    const float ref = reference(top);
    unsigned long long s2 = 0ull;
    const unsigned long long c2 = pack2(c, c);
    const float rc = -__fmul_rn(ref, c);
    if (plain_product(rc)) {
      const unsigned long long rc2 = pack2(rc, rc);
      for (int i = tid; i < v1 - v0; i += kDistillThreads) {
        float o[W];
        unpack(vec_held[i], o, T{});
#pragma unroll
        for (int j = 0; j < W; j += 2) {
          const float2 d = unpack2(fma2(pack2(o[j], o[j + 1]), c2, rc2));
          s2 = add2(s2, pack2(exp2_approx(d.x), exp2_approx(d.y)));
        }
      }
    } else {
      for (int i = tid; i < v1 - v0; i += kDistillThreads) {
        float o[W];
        unpack(vec_held[i], o, T{});
#pragma unroll
        for (int j = 0; j < W; ++j) s2 = add2(s2, pack2(exp2_approx(exponent(o[j], ref, c)), 0.0f));
      }
    }
    float rest = unpack2(s2).x + unpack2(s2).y, in = 0.0f;
    // the warp's maxima, edges and ids with them, and its sums against these; without
    // the class for the rest only the whole row's sum is wanted, and `rest` is that
    const bool edge_apart = apart && edge_in;
    float rest_m = warp_max(fmaxf(fmaxf(top, edge_apart ? -INFINITY : edge), apart ? -INFINITY : in_m));
    float ids_m = apart ? warp_max(fmaxf(in_m, edge_apart ? edge : -INFINITY)) : -INFINITY;
    rest = move_sum(rest, top, rest_m, c);
    if (edge_i >= 0) (edge_apart ? in : rest) += exp2_approx(exponent(edge, reference(edge_apart ? ids_m : rest_m), c));
    if (own >= 0 && !again) (apart ? in : rest) += exp2_approx(exponent(mine, reference(apart ? ids_m : rest_m), c));
    for (int o = 16; o > 0; o >>= 1) {
      rest += __shfl_xor_sync(0xffffffffu, rest, o);
      if (apart) in += __shfl_xor_sync(0xffffffffu, in, o);
    }
    if (lane == 0) {
      sh.rest_m[warp] = rest_m;
      sh.rest[warp] = rest;
      sh.in_m[warp] = ids_m;
      sh.in[warp] = in;
    }
    __syncthreads();
    // the lanes' sums onto the maxima of all lanes, and their sums, in every lane
    auto join = [&](bool have, const float *m_rest, const float *s_rest, const float *m_in, const float *s_in) {
      const float of = have ? m_rest[lane] : -INFINITY, of_in = have && apart ? m_in[lane] : -INFINITY;
      rest = have ? s_rest[lane] : 0.0f;        // lanes without one add 0
      in = have && apart ? s_in[lane] : 0.0f;
      rest_m = warp_max(of);
      if (apart) ids_m = warp_max(of_in);
      rest = move_sum(rest, of, rest_m, c);
      in = move_sum(in, of_in, ids_m, c);
      for (int o = 16; o > 0; o >>= 1) {
        rest += __shfl_xor_sync(0xffffffffu, rest, o);
        if (apart) in += __shfl_xor_sync(0xffffffffu, in, o);
      }
    };
    join(lane < kDistillWarps, sh.rest_m, sh.rest, sh.in_m, sh.in);   // the CTA's, in every thread
    cluster_wait();                       // every CTA of the cluster has started
    if (tid < static_cast<int>(cs)) {     // to every CTA, so that all go on with the same bits
      peer_store32(peer_addr(&sh.from_rest_m[cr], tid), __float_as_uint(rest_m));
      peer_store32(peer_addr(&sh.from_rest[cr], tid), __float_as_uint(rest));
      if (apart) {
        peer_store32(peer_addr(&sh.from_in_m[cr], tid), __float_as_uint(ids_m));
        peer_store32(peer_addr(&sh.from_in[cr], tid), __float_as_uint(in));
      }
    }
    if (own >= 0) peer_store32(peer_addr(&sh.x[tid], 0), __float_as_uint(mine));
    if (edge_in)
      for (int j = 0; j < k; ++j)
        if (sh.id[j] == edge_i) peer_store32(peer_addr(&sh.x[j], 0), __float_as_uint(edge));
    cluster_sync();

    join(lane < static_cast<int>(cs), sh.from_rest_m, sh.from_rest, sh.from_in_m, sh.from_in);
    const float most = fmaxf(rest_m, ids_m), mass = sh.mass;
    const float total = apart ? move_sum(rest, rest_m, most, c) + move_sum(in, ids_m, most, c) : rest;
    // all masked (the sums stay 0), or NaN beside masked values: against 0
    const float m = reference(most), mr = reference(rest_m);
    const float pt = a.tail ? left_over(mass) : 0.0f;
    if (cr == 0 && warp == 0 && a.loss) {
      // a few values a row, in 64 bits: a lowest value would overflow in log2's units
      // Differences of logits first: of 3.4e38 in size they would swallow the sum's logarithm.
      const double log_sum = row_log_sum(m, c, log2f(total));
      double loss = 0.0;
      for (int j = lane; j < k; j += 32)
        if (sh.p[j] != 0.0f)              // NaNs too
          loss += sh.p[j] * (sh.lp[j] - ((static_cast<double>(sh.x[j]) - m) * a.inv_temperature64 - log_sum));
      for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
      if (pt > 0.0f)
        loss += pt * (logf(pt) - ((static_cast<double>(mr) - m) * a.inv_temperature64 +
                                  row_log_sum(mr, c, log2f(rest)) - log_sum));
      if (lane == 0) a.loss[row] = total == 0.0f ? 0.0f : static_cast<float>(w * loss);
    }
    if (total == 0.0f) {
      scale = 0.0f;
    } else {
      const float q = (mass + pt) / total;
      f_in = q * scale;
      f_out = !apart ? f_in : rest == 0.0f ? 0.0f : (q * exp2_approx(shift_exponent(mr, m, c)) - pt / rest) * scale;
    }
    if (!g) return;
    if (own >= 0) {
      if (again) {
        own = -1;                         // the first entry of the id writes for all
      } else {
        float r = sh.p[tid];
        if (sh.twice[0] | sh.twice[1])
          for (int j = tid + 1; j < k; ++j)
            if (sh.id[j] == first + own) r += sh.p[j];
        in_m = exp2_approx(exponent(mine, m, c)) * f_in - r * scale;
      }
    }
    if (edge_i >= 0) {
      const float e = exp2_approx(exponent(edge, edge_in ? m : mr, c));
      if (edge_in) {
        float r = 0.0f;
        for (int j = 0; j < k; ++j)
          if (sh.id[j] == edge_i) r += sh.p[j];
        edge = e * f_in - r * scale;
      } else {
        edge = e * f_out;
      }
    }
    if (scale == 0.0f) edge = in_m = 0.0f;
    top = in_m;
    // the gradient outside S; the ids' places are 0 here (-infinity in the row)
    if (scale != 0.0f) {
      const float rc = -__fmul_rn(mr, c);
      if (plain_product(rc) && (reinterpret_cast<uintptr_t>(g + first) & 15) == 0) {
        uint4 *gv = reinterpret_cast<uint4 *>(g + first);
        const unsigned long long rc2 = pack2(rc, rc), f2 = pack2(f_out, f_out);
        for (int i = tid; i < v1 - v0; i += kDistillThreads) {
          float o[W];
          unpack(vec_held[i], o, T{});
          float r[W];
#pragma unroll
          for (int j = 0; j < W; j += 2) {
            const float2 d = unpack2(fma2(pack2(o[j], o[j + 1]), c2, rc2));
            const float2 q = unpack2(mul2(pack2(exp2_approx(d.x), exp2_approx(d.y)), f2));
            r[j] = q.x;
            r[j + 1] = q.y;
          }
          __stcs(gv + i, pack_vec(r, T{}));
        }
      } else {                            // rows of another alignment than the logits', or of lowest values
        for (int i = tid; i < count; i += kDistillThreads)
          g[first + i] = from_float<T>(exp2_approx(exponent(to_float(row_held[i]), mr, c)) * f_out);
      }
      __syncthreads();                    // the zeros at the ids' places are written
      if (own >= 0) g[first + own] = from_float<T>(top);
      if (edge_i >= 0) g[edge_i] = from_float<T>(edge);
      return;
    }
  } else {
    cluster_wait();
    if (cr == 0 && tid == 0 && a.loss) a.loss[row] = 0.0f;
    if (!g) return;
  }
  // no weight, or nothing above -infinity: zeros
  for (int i = tid; i < count; i += kDistillThreads) g[first + i] = from_float<T>(0.0f);
  if (edge_i >= 0) g[edge_i] = from_float<T>(0.0f);
}

__device__ __forceinline__ float block_sum(float v, float *s) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.0f;
  for (int w = 0; w < kDistillThreads / 32; ++w) r += s[w];
  return r;
}

// One CTA a row, read once for the maximum, once for the sums and once for the
// gradient: rows that a cluster's shared memory cannot hold.
template <typename T>
__global__ void __launch_bounds__(kDistillThreads) distill_long_kernel(const DistillArgs a) {
  __shared__ float s_red[kDistillThreads / 32];
  __shared__ float s_max[kDistillThreads / 32];
  __shared__ int s_id[kMaxTop];
  __shared__ float s_x[kMaxTop], s_p[kMaxTop];
  __shared__ uint32_t s_seen[64];                      // 2,048 bits: ids mod 2,048
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  T *g = a.grad ? static_cast<T *>(a.grad) + row * a.grad_ld : nullptr;
  const int tid = threadIdx.x;
  const uint32_t v = static_cast<uint32_t>(a.v);       // below 2^31: a step past it stays a uint32_t
  const float inv_t = a.inv_temperature;
  const float w = a.row_weight ? a.row_weight[row] : 1.0f;

  if (tid < 64) s_seen[tid] = 0u;
  __syncthreads();
  if (tid < a.n_top) {
    const int id = a.teacher_ids[row * a.n_top + tid];
    const bool ok = id >= 0 && static_cast<uint32_t>(id) < v;
    s_id[tid] = ok ? id : -1;
    s_p[tid] = ok ? a.teacher_logprobs[row * a.n_top + tid] : -INFINITY;
    s_x[tid] = ok ? to_float(x[id]) : -INFINITY;
    if (ok) atomicOr(&s_seen[(id & 2047) >> 5], 1u << (id & 31));
  }
  __syncthreads();
  auto named = [&](uint32_t i) {
    if (!((s_seen[(i & 2047) >> 5] >> (i & 31)) & 1u)) return false;
    for (int j = 0; j < a.n_top; ++j)
      if (s_id[j] == static_cast<int>(i)) return true;
    return false;
  };
  // maxima and sums outside the ids and of the ids, as in distill_kernel
  float rest_m = -INFINITY, ids_m = -INFINITY;
  for (uint32_t i = tid; i < v; i += kDistillThreads)
    if (!named(i)) rest_m = fmaxf(rest_m, to_float(x[i]));
  rest_m = warp_max(rest_m);
  if ((tid & 31) == 0) s_max[tid >> 5] = rest_m;
  __syncthreads();
  for (int i = 0; i < kDistillThreads / 32; ++i) rest_m = fmaxf(rest_m, s_max[i]);
  for (int j = 0; j < a.n_top; ++j) ids_m = fmaxf(ids_m, s_x[j]);
  const float mr = reference(rest_m), mi = reference(ids_m), m = reference(fmaxf(rest_m, ids_m));
  float rest = 0.0f, in = 0.0f;
  for (uint32_t i = tid; i < v; i += kDistillThreads) {
    if (named(i)) in += expf((to_float(x[i]) - mi) * inv_t);
    else rest += expf((to_float(x[i]) - mr) * inv_t);
  }
  rest = block_sum(rest, s_red);
  in = block_sum(in, s_red);
  auto moved = [&](float s, float from) { return s == 0.0f ? s : s * expf((from - m) * inv_t); };   // a NaN stays one
  const float total = moved(rest, rest_m) + moved(in, ids_m), logs = logf(total);
  if (w == 0.0f || total == 0.0f) {                    // no weight, or a row without a distribution
    if (tid == 0 && a.loss) a.loss[row] = 0.0f;
    if (g)
      for (uint32_t i = tid; i < v; i += kDistillThreads) g[i] = from_float<T>(0.0f);
    return;
  }

  float lmax = -INFINITY, mass = 0.0f;
  double loss = 0.0;                                   // as in distill_kernel
  for (int j = 0; j < a.n_top; ++j) lmax = fmaxf(lmax, s_p[j]);
  float logsum = 0.0f;
  if (a.tail || lmax == -INFINITY) {
    lmax = 0.0f;
  } else {
    float sum = 0.0f;
    for (int j = 0; j < a.n_top; ++j) sum += expf(s_p[j] - lmax);
    logsum = logf(sum);
  }
  for (int j = 0; j < a.n_top; ++j) {
    const float lp = s_p[j] - lmax - logsum, p = expf(lp);
    mass += p;
    if (p != 0.0f) loss += p * (lp - ((static_cast<double>(s_x[j]) - m) * a.inv_temperature64 - logs));
  }
  __syncthreads();
  if (tid < a.n_top) s_p[tid] = expf(s_p[tid] - lmax - logsum);
  const float pt = a.tail ? left_over(mass) : 0.0f;
  if (pt > 0.0f) loss += pt * (logf(pt) - ((static_cast<double>(mr) - m) * a.inv_temperature64 + logf(rest) - logs));
  if (tid == 0 && a.loss) a.loss[row] = static_cast<float>(w * loss);
  if (!g) return;
  __syncthreads();
  const float scale = w * inv_t;
  const float f_in = (mass + pt) / total * scale;
  const float f_out = rest != 0.0f ? ((mass + pt) / total * expf((mr - m) * inv_t) - pt / rest) * scale : 0.0f;
  for (uint32_t i = tid; i < v; i += kDistillThreads) {
    float r;
    if (!named(i)) {
      r = expf((to_float(x[i]) - mr) * inv_t) * f_out;
    } else {
      r = expf((to_float(x[i]) - m) * inv_t) * f_in;
      for (int j = 0; j < a.n_top; ++j)
        if (s_id[j] == i) r -= s_p[j] * scale;
    }
    g[i] = from_float<T>(r);
  }
}

template <typename T>
cudaError_t launch_distill_long(const DistillArgs &a) {
  distill_long_kernel<T><<<static_cast<unsigned>(a.n), kDistillThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_distill_t(const DistillArgs &a) {
  static std::atomic<unsigned long long> configured{0};   // one bit per device; host threads may race here
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(distill_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(distill_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldOne);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  // As few CTAs as hold the row four to an SM (1,024 bf16 rows of 202,048: 166 us,
  // against 194 us three to an SM and 266 us eight of half the share), more while there are SMs to fill;
  // 16 with fewer to an SM for the longest rows.
  const int64_t bytes = a.v * static_cast<int64_t>(sizeof(T));
  auto held = [&](int64_t cs) { return (bytes / 16 + cs - 1) / cs * 16; };   // a share is at most this
  int cs = 1;
  while (cs < kDistillCluster && held(cs) > kHeldFour) cs *= 2;
  while (cs < kDistillCluster && a.n * 2 * cs <= 2 * a.num_sms && a.v / (2 * cs) >= 2048) cs *= 2;
  if (held(cs) > kHeldOne) return launch_distill_long<T>(a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n * cs));
  cfg.blockDim = dim3(kDistillThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(held(cs));
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start before the previous grid ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (held(cs) > kHeldFour) {             // up to 16 SMs of one GPC at a time: not every device has them
    int fit = 0;
    e = cudaOccupancyMaxActiveClusters(&fit, distill_kernel<T>, &cfg);
    if (e != cudaSuccess) return e;
    if (fit < 1) return launch_distill_long<T>(a);
  }
  return cudaLaunchKernelEx(&cfg, distill_kernel<T>, a);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs &a) {
  if (a.dtype == 0) return launch_distill_t<float>(a);
  if (a.dtype == 1) return launch_distill_t<__half>(a);
  return launch_distill_t<__nv_bfloat16>(a);
}

}  // namespace muse
