// Device helpers of the training-objective operators (k_topk.cu, k_distill.cu,
// k_route.cu): rows of bf16, fp16 or fp32 logits read in 16-byte vectors.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/scape.h"
#include "scape_device.cuh"

namespace scape {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

// 2^x, relative error below 2^-22 (PTX ex2.approx); 2^-inf = +0, NaN stays NaN.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16-byte load of a row that is read once.  Not the read-only path: a gradient
// may overwrite the logits in the same kernel.
__device__ __forceinline__ uint4 ld_row_u4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// 1 / x, off by at most one unit in the last place.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values: one instruction for two operations.
using pair_t = float2;
__device__ __forceinline__ pair_t pair(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ pair_t ex2_2(pair_t v) { return pair(ex2(v.x), ex2(v.y)); }

// Thread-block clusters: this CTA's place, the barrier over all their threads
// (it orders memory), and stores to another CTA's shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// (for threads that have written nothing that others read)
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address in CTA "rank" of what lies at "local" in this one.
__device__ __forceinline__ uint32_t remote_at(const void* local, uint32_t rank) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(local);
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  return there;
}
__device__ __forceinline__ void put_remote(const float* local, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote_at(local, rank)), "f"(v) : "memory");
}
__device__ __forceinline__ void put_remote(const uint64_t* local, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote_at(local, rank)), "l"(v) : "memory");
}

// Asynchronous 16-byte copy to shared memory.  A thread that reads back only
// what it copied itself needs no barrier, only its own wait.
__device__ __forceinline__ void copy_async(uint32_t smem, const void* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(p) : "memory");
}
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// A maximum as the shift of a softmax: exp2((x - m) * c) of a row that holds
// nothing but -inf is then exp2(-inf) = 0 and not NaN.
__device__ __forceinline__ float shift_of(float m) { return m == neg_inf() ? 0.0f : m; }

// The terms 2^((x - m) c) of such a sum at one FMA each, as 2^(x c' - k).  In
// general c' = c and k = m c rounded: the FMA takes the exact product, so the
// terms are all off by the same factor 2^(m c - k), which fix takes out of their
// sum.  That holds while the factor is within 2^32, for m c below 2^30.  Beyond,
// what is below m is so by 32 / c at least and its term is 0 in fp32; any c' shows
// that, and with a power of two that puts m c' between 2^31 and 2^32 k is exact,
// and finite down to the type's lowest value.  m is finite (+inf gives NaN).
struct Shift {
  float c, k;
  __device__ __forceinline__ Shift(float m, float c_) : c(c_), k(m * c_) {
    if (!(fabsf(k) < 0x1p30f)) {
      const int biased = (__float_as_int(m) >> 23) & 0xFF;
      c = __int_as_float(min(285 - biased, 254) << 23);
      k = m * c;
    }
  }
  __device__ __forceinline__ float term(float x) const { return ex2(__fmaf_rn(x, c, -k)); }
  __device__ __forceinline__ float fix(float m) const { return ex2(__fmaf_rn(-m, c, k)); }
};

// 2^((x - m) c) for two logits: in one FMA by Shift, whose few instructions a row
// pay off over many vectors, or as a difference and a product (DIFF), which is
// the faster one where a thread has a vector or two.
template <bool DIFF>
struct Terms {
  pair_t c, k;
  float undo = 1.0f;  // Shift's fix()
  __device__ __forceinline__ Terms(float m, float c_) : c(pair(c_, c_)), k(pair(-m, -m)) {
    if (DIFF) return;
    const Shift by(m, c_);
    c = pair(by.c, by.c);
    k = pair(-by.k, -by.k);
    undo = by.fix(m);
  }
  __device__ __forceinline__ pair_t operator()(pair_t x) const {
    return ex2_2(DIFF ? mul2(add2(x, k), c) : fma2(x, c, k));
  }
};

template <int DT>
struct Elem;

template <>
struct Elem<SCAPE_BF16> {
  using T = uint16_t;
  static constexpr int kPerVec = 8;
  static __device__ __forceinline__ float load(const T* p) { return bf16f(*p); }
  static __device__ __forceinline__ T make(float f) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  }
  static __device__ __forceinline__ void unpack(const uint4 r, float (&f)[8]) {
    f[0] = bf16lo(r.x); f[1] = bf16hi(r.x); f[2] = bf16lo(r.y); f[3] = bf16hi(r.y);
    f[4] = bf16lo(r.z); f[5] = bf16hi(r.z); f[6] = bf16lo(r.w); f[7] = bf16hi(r.w);
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
  static constexpr uint32_t kNegInf2 = 0xFF80FF80u;  // two lowest elements
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 h = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                     *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <>
struct Elem<SCAPE_F16> {
  using T = uint16_t;
  static constexpr int kPerVec = 8;
  static __device__ __forceinline__ float load(const T* p) {
    return __half2float(__ushort_as_half(*p));
  }
  static __device__ __forceinline__ T make(float f) { return __half_as_ushort(__float2half_rn(f)); }
  static __device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = t.x;
    b = t.y;
  }
  static __device__ __forceinline__ void unpack(const uint4 r, float (&f)[8]) {
    unpack2(r.x, f[0], f[1]); unpack2(r.y, f[2], f[3]);
    unpack2(r.z, f[4], f[5]); unpack2(r.w, f[6], f[7]);
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
  static constexpr uint32_t kNegInf2 = 0xFC00FC00u;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __half2 h = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <>
struct Elem<SCAPE_F32> {
  using T = float;
  static constexpr int kPerVec = 4;
  static __device__ __forceinline__ float load(const T* p) { return *p; }
  static __device__ __forceinline__ T make(float f) { return f; }
  static __device__ __forceinline__ void unpack(const uint4 r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static constexpr uint32_t kNegInf2 = 0xFF800000u;  // (one element)
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
};

// Whether all elements of a vector are below a bound of the same type (NaN is
// not; the bound comes in both halves of a word for 16-bit elements).
template <int DT>
__device__ __forceinline__ bool all_below(const uint4 v, uint32_t bound) {
  if constexpr (DT == SCAPE_BF16) {
    auto h = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h(v.x), h(v.y)), __hmax2_nan(h(v.z), h(v.w)));
    return __hblt2(m, h(bound));
  } else if constexpr (DT == SCAPE_F16) {
    auto h = [](uint32_t x) { return *reinterpret_cast<const __half2*>(&x); };
    const __half2 m = __hmax2_nan(__hmax2_nan(h(v.x), h(v.y)), __hmax2_nan(h(v.z), h(v.w)));
    return __hblt2(m, h(bound));
  } else {
    const float b = __uint_as_float(bound);
    return __uint_as_float(v.x) < b && __uint_as_float(v.y) < b && __uint_as_float(v.z) < b &&
           __uint_as_float(v.w) < b;
  }
}
// The largest element not above f, as all_below() takes it.
template <int DT>
__device__ __forceinline__ uint32_t bound_of(float f) {
  if constexpr (DT == SCAPE_BF16) {
    const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rd(f));
    return h << 16 | h;
  } else if constexpr (DT == SCAPE_F16) {
    const uint32_t h = __half_as_ushort(__float2half_rd(f));
    return h << 16 | h;
  } else {
    return __float_as_uint(f);
  }
}

// Element by element the larger one of two vectors (NaN loses).
template <int DT>
__device__ __forceinline__ uint4 max_vec(const uint4 a, const uint4 b) {
  using E = Elem<DT>;
  return make_uint4(E::max2(a.x, b.x), E::max2(a.y, b.y), E::max2(a.z, b.z), E::max2(a.w, b.w));
}
template <int DT>
__device__ __forceinline__ uint4 neg_inf_vec() {
  constexpr uint32_t n = Elem<DT>::kNegInf2;
  return make_uint4(n, n, n, n);
}

// One row seen as 16-byte vectors on 16-byte boundaries.  A row starts at any
// element (odd vocabularies, views): vector v holds the elements
// [v * kPerVec - shift, + kPerVec), and those outside [0, n) read as -inf.
template <int DT>
struct RowView {
  using E = Elem<DT>;
  using T = typename E::T;
  const T* p;
  int64_t n;
  int shift;
  __device__ __forceinline__ RowView(const void* base, int64_t first, int64_t len)
      : p(static_cast<const T*>(base) + first), n(len) {
    shift = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  }
  __device__ __forceinline__ int64_t vectors() const {
    return (n + shift + E::kPerVec - 1) / E::kPerVec;
  }
  __device__ __forceinline__ int64_t first_of(int64_t v) const { return v * E::kPerVec - shift; }
  __device__ __forceinline__ uint4 load(int64_t v) const {
    const int64_t e = first_of(v);
    if (e >= 0 && e + E::kPerVec <= n) return ld_row_u4(p + e);
    float f[E::kPerVec];
#pragma unroll
    for (int j = 0; j < E::kPerVec; j++)
      f[j] = (e + j >= 0 && e + j < n) ? E::load(p + e + j) : neg_inf();
    return E::pack(f);
  }
};

// Ordered key of a logit: unsigned comparison ranks as the values do, +0 and
// -0 alike, NaN above +inf.  No logit has key 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// ... and the logit of a key (of zero +0, of NaN one of them).
__device__ __forceinline__ float value_of_key(uint32_t k) {
  return k == 0xFFFFFFFFu ? __uint_as_float(0x7FFFFFFFu)
                          : __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Sum / maximum over the CTA; every thread receives it.  "buf" is shared
// scratch of 32 entries; the calls contain two __syncthreads().
template <class V>
__device__ __forceinline__ V cta_sum(V x, V* buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  x = lane < nw ? buf[lane] : V(0);
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

__device__ __forceinline__ float cta_max(float x, float* buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  x = lane < nw ? buf[lane] : neg_inf();
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}

}  // namespace scape
