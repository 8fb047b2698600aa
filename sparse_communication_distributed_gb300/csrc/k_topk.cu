// The k largest logits of every row, in order, and the row's log-sum-exp: what
// a teacher leaves behind for distillation.
//
// Candidates are ranked by the unique composite key << 32 | ~index (order_key
// of objective.cuh), so that equal logits go to the lower index.  A CTA takes a
// row in tiles that its threads hold in registers.  Of each tile it keeps the
// elements above the k-th best so far; if those are too many for the list in
// shared memory, a search by bits finds the tile's own k-th best first (every
// step counts the elements above a bound).  The list is sorted and cut to k
// after each tile.  The same pass carries a running maximum and sum of
// exponentials in every thread.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "objective.cuh"
#include "scape_kernels.cuh"

#define SCAPE_API extern "C" __attribute__((visibility("default")))

namespace scape {
namespace {

constexpr int kThreads = 512;
constexpr int kVecs = 8;     // vectors a thread holds of a tile
constexpr int kMaxK = 1024;
constexpr int kCap = 2 * kMaxK;  // list entries: the k best so far and k new ones always fit

struct TopkArgs {
  const void* x;
  int64_t rows, V, stride;
  int k;
  float tau, c;  // temperature, log2(e) / temperature
  int32_t* idx;
  void* vals;
  float* lse;
};

// Sorts list[0..n) in descending order (bitonic, padded with 0).
__device__ void sort_list(uint64_t* list, int n) {
  int P = 1;
  while (P < n) P <<= 1;
  for (int i = n + threadIdx.x; i < P; i += kThreads) list[i] = 0;
  for (int size = 2; size <= P; size <<= 1)
    for (int d = size >> 1; d; d >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < P / 2; i += kThreads) {
        const int lo = (i / d) * 2 * d + (i % d), hi = lo + d;
        const bool up = (lo & size) != 0;
        const uint64_t a = list[lo], b = list[hi];
        if ((a < b) != up) {
          list[lo] = b;
          list[hi] = a;
        }
      }
    }
  __syncthreads();
}

template <int DT>
__global__ __launch_bounds__(kThreads) void topk_rows(const TopkArgs a) {
  using E = Elem<DT>;
  constexpr int EPV = E::kPerVec;
  __shared__ uint64_t list[kCap];
  __shared__ uint32_t ubuf[32];
  __shared__ float fbuf[32];
  __shared__ uint32_t n_shared;
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const RowView<DT> view(a.x, row * a.stride, a.V);
    const int64_t nv = view.vectors();
    uint32_t n = 0;
    uint64_t thr = 0;  // composites have to exceed it
    float m = neg_inf(), s = 0.0f;
    for (int64_t t0 = 0; t0 < nv; t0 += kThreads * kVecs) {
      uint4 r[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; i++) {
        const int64_t v = t0 + i * kThreads + tid;
        r[i] = v < nv ? view.load(v) : make_uint4(E::kNegInf2, E::kNegInf2, E::kNegInf2, E::kNegInf2);
      }
      auto each = [&](auto f) {
#pragma unroll 1
        for (int i = 0; i < kVecs; i++) {
          uint4 q = r[0];
#pragma unroll
          for (int u = 1; u < kVecs; u++) q = i == u ? r[u] : q;
          float x[EPV];
          E::unpack(q, x);
          const int64_t e0 = view.first_of(t0 + i * kThreads + tid);
#pragma unroll
          for (int j = 0; j < EPV; j++)
            if (e0 + j >= 0 && e0 + j < view.n) f(x[j], (uint32_t)(e0 + j));
        }
      };
      auto comp = [](float x, uint32_t e) { return (uint64_t)order_key(x) << 32 | (uint32_t)~e; };
      auto count_from = [&](uint64_t lo) {  // elements above thr and not below lo
        uint32_t c = 0;
        each([&](float x, uint32_t e) {
          const uint64_t v = comp(x, e);
          c += v > thr && v >= lo;
        });
        return cta_sum(c, ubuf);
      };
      // running maximum and sum of exponentials
      float mt = m;
      each([&](float x, uint32_t) { mt = fmaxf(mt, x); });
      s *= ex2((shift_of(m) - shift_of(mt)) * a.c);
      m = mt;
      const float sh = shift_of(m);
      each([&](float x, uint32_t) { s += ex2((x - sh) * a.c); });
      // the elements to list: all above thr, or the tile's own k best
      uint64_t cut = 0;
      uint32_t c = count_from(0);
      if (n + c > kCap) {
        for (int b = 63; b >= 0; b--) {
          const uint64_t t = cut | (1ull << b);
          c = count_from(t);
          if (c >= (uint32_t)a.k) cut = t;
          if (c >= (uint32_t)a.k && n + c <= kCap) break;
        }
      }
      if (tid == 0) n_shared = n;
      __syncthreads();
      each([&](float x, uint32_t e) {
        const uint64_t v = comp(x, e);
        if (v > thr && v >= cut) list[atomicAdd(&n_shared, 1u)] = v;
      });
      __syncthreads();
      n = n_shared;
      sort_list(list, (int)n);
      if (n >= (uint32_t)a.k) {
        n = a.k;
        thr = list[n - 1];
      }
      __syncthreads();
    }
    for (int i = tid; i < a.k; i += kThreads) {
      const int32_t e = (int32_t)~(uint32_t)list[i];
      a.idx[row * a.k + i] = e;
      if (a.vals) static_cast<typename E::T*>(a.vals)[row * a.k + i] = view.p[e];
    }
    if (a.lse) {
      const float M = cta_max(m, fbuf), sh = shift_of(M);
      const float S = cta_sum(s * ex2((shift_of(m) - sh) * a.c), fbuf);
      if (tid == 0) a.lse[row] = sh / a.tau + logf(S);
    }
    __syncthreads();
  }
}

int fail(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_thread_error(buf);
  return code;
}

}  // namespace
}  // namespace scape

SCAPE_API int scape_topk_logits(const void* logits, int dtype, uint64_t rows, uint64_t vocab,
                                uint64_t row_stride, int k, float temperature, int32_t* idx,
                                void* vals, float* lse, void* stream) {
  using namespace scape;
  if (dtype < SCAPE_BF16 || dtype > SCAPE_F32) return fail(SCAPE_EINVAL, "unknown dtype %d", dtype);
  if (vocab < 1 || vocab >= (1ull << 31))
    return fail(SCAPE_EINVAL, "vocab=%llu must be in [1, 2^31)", (unsigned long long)vocab);
  if (k < 1 || k > kMaxK || (uint64_t)k > vocab)
    return fail(SCAPE_EINVAL, "k=%d outside [1, min(vocab, %d)]", k, kMaxK);
  if (row_stride < vocab) return fail(SCAPE_EINVAL, "row_stride must be >= vocab");
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(kLog2e / temperature))
    return fail(SCAPE_EINVAL, "temperature must be finite and > 0");
  if (rows >= (1ull << 31) || row_stride >= (1ull << 32))
    return fail(SCAPE_EINVAL, "rows must be < 2^31 and row_stride < 2^32");
  if (rows == 0) return SCAPE_OK;
  if (!logits || !idx) return fail(SCAPE_EINVAL, "logits and idx are required");
  const uintptr_t es = dtype == SCAPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(vals) % es ||
      reinterpret_cast<uintptr_t>(idx) % 4 || reinterpret_cast<uintptr_t>(lse) % 4)
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  TopkArgs a{};
  a.x = logits;
  a.rows = (int64_t)rows;
  a.V = (int64_t)vocab;
  a.stride = (int64_t)row_stride;
  a.k = k;
  a.tau = temperature;
  a.c = kLog2e / temperature;
  a.idx = idx;
  a.vals = vals;
  a.lse = lse;
  const uint64_t cap = (uint64_t)num_sms() * 2;
  const unsigned grid = (unsigned)(rows < cap ? rows : cap);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SCAPE_BF16) topk_rows<SCAPE_BF16><<<grid, kThreads, 0, s>>>(a);
  else if (dtype == SCAPE_F16) topk_rows<SCAPE_F16><<<grid, kThreads, 0, s>>>(a);
  else topk_rows<SCAPE_F32><<<grid, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "topk_rows: %s", cudaGetErrorString(e));
}
