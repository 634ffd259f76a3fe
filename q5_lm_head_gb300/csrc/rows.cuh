// Helpers of the kernels that read rows of logits in 32 or 16 bits (score.cu,
// distill.cu): conversions, a row's cut into 16-byte vectors, sums over a
// cluster's shared memory.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace muse {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The values of a 16-byte vector.
template <typename T>
struct Vec {
  static constexpr int W = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4 &r, float (&o)[4], float) {
  o[0] = __uint_as_float(r.x);
  o[1] = __uint_as_float(r.y);
  o[2] = __uint_as_float(r.z);
  o[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint4 &r, float (&o)[8], __half) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    o[2 * i] = f.x;
    o[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack(const uint4 &r, float (&o)[8], __nv_bfloat16) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(w[i] << 16);
    o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack_vec(const float (&o)[4], float) {
  return make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3]));
}
__device__ __forceinline__ uint4 pack_vec(const float (&o)[8], __half) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(o[2 * i], o[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack_vec(const float (&o)[8], __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Maxima of vectors, value by value; a NaN yields to the other value.
__device__ __forceinline__ uint4 vec_lowest(float) { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
__device__ __forceinline__ uint4 vec_lowest(__half) { return make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u); }
__device__ __forceinline__ uint4 vec_lowest(__nv_bfloat16) { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b, float) {
  return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b, __half) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ uint4 vec_max(const uint4 &a, const uint4 &b, T t) {
  return make_uint4(max_word(a.x, b.x, t), max_word(a.y, b.y, t), max_word(a.z, b.z, t), max_word(a.w, b.w, t));
}

// A row of v values as `head` values before the first 16-byte boundary, `vecs`
// aligned vectors and the rest: rows may start at any element.
struct RowCut {
  int head, vecs;
};
template <typename T>
__device__ __forceinline__ RowCut cut_row(const T *x, int v) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15) / static_cast<int>(sizeof(T));
  int head = off ? Vec<T>::W - off : 0;
  if (head > v) head = v;
  return {head, (v - head) / Vec<T>::W};
}

// The float of a float_order_key.
__device__ __forceinline__ float order_key_float(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// 2 ulp, 0 below the smallest normal: as good as expf to a sum of a row's
// exponentials, which is off by more for its additions, and one instruction, of
// which these kernels have few to spare beside their loads.
__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Two f32 values in one 64-bit register: one instruction works on both.
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// (x - m) c, c = log2(e) / temperature: the exponent of x against the row's
// reference m.  One fma with the rounded product m c as the reference itself,
// which every use of it shares.  The rounding moves the reference by up to
// 2^-24 |m c|: below 2^20 by a sixteenth, but for masks of -1e10 by hundreds, which
// would leave no value of the row in range.  From there on the difference is
// taken first, and the reference is m c itself.
constexpr float kPlain = 1048576.0f;
__device__ __forceinline__ bool plain_product(float mc) { return fabsf(mc) < kPlain; }   // of no infinity or NaN
__device__ __forceinline__ float exponent(float x, float m, float c) {
  const float mc = __fmul_rn(m, c);
  return plain_product(mc) ? fmaf(x, c, -mc) : (x - m) * c;
}
// What m c is above its reference.
__device__ __forceinline__ float reference_off(float m, float c) {
  const float mc = __fmul_rn(m, c);
  return plain_product(mc) ? fmaf(m, c, -mc) : 0.0f;
}
// The exponent by which sums against reference `from` move to reference `to`.
__device__ __forceinline__ float shift_exponent(float from, float to, float c) {
  const float f = __fmul_rn(from, c), t = __fmul_rn(to, c);
  if (plain_product(f) && plain_product(t)) return __fadd_rn(f, -t);
  return (from - to) * c - reference_off(from, c) + reference_off(to, c);
}

// log sum exp((x - m) / temperature) from log2 of the sum of exponents against m, in
// 64 bits.  The logarithm against m itself takes off again what the reference
// was beside it.
constexpr double kLn2 = 0.6931471805599453;
__device__ __forceinline__ double row_log_sum(float m, float c, float log2_sum) {
  return kLn2 * (static_cast<double>(log2_sum) - reference_off(m, c));
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster; orders shared-memory accesses
// before it, the distributed ones too, against those after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same in two halves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of p (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return a;
}
__device__ __forceinline__ void peer_store64(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void peer_store32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

}  // namespace muse
