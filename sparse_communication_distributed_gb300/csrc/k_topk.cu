// The k largest logits of every row, in order, and the row's log-sum-exp: what
// a teacher leaves behind for distillation.
//
// Candidates are ranked by the unique composite key << 32 | ~index (order_key
// of objective.cuh), so that equal logits go to the lower index.  A CTA takes a
// row in tiles of up to 64 KB of shared memory; each thread works on vectors
// that it copied itself.  One pass over a tile keeps, for each of G groups of
// elements (a group is one place or a few of the vectors that a thread sees),
// the group's largest element so far.  At least k elements reach the k-th
// largest of these G, so nothing below it is among the row's k best; a histogram
// of the G over their range gives a bound just under it.  A second pass lists
// what reaches the bound -- for logits in no special order k (1 + k / 2G)
// elements of a first tile, a t-th part of that of the t-th tile -- and sums the
// exponentials.  The list is sorted in the end.  Where too much reaches the
// bound (many equal logits, few above -inf, adverse orders), the tile is read
// again and its own k-th best composite is found bit by bit.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "objective.cuh"
#include "scape_kernels.cuh"

#define SCAPE_API extern "C" __attribute__((visibility("default")))

namespace scape {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 16;  // vectors a thread has of a tile
constexpr int kTile = kThreads * kVecs;
constexpr int kBlk = 2;    // vectors a thread handles at a time
constexpr int kMaxK = 1024;
constexpr int kBins = 256;
constexpr int kHits = 1024;
constexpr int kCountSort = 256;  // lists up to this are sorted by counting

struct TopkArgs {
  const void* x;
  int64_t rows, V, stride;
  int k;
  int cap;          // list entries; k of an earlier tile and k new ones always fit
  int tile;         // vectors of a tile
  float tau, c;     // temperature, log2(e) / temperature
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
        const int lo = (i & ~(d - 1)) * 2 + (i & (d - 1)), hi = lo + d;
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

// GROUPS: groups of a thread (1, 2, 4 or 8 for 16-bit elements, up to 4 else).
template <int DT, int GROUPS>
__global__ __launch_bounds__(kThreads, 3) void topk_rows(const TopkArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int EPV = E::kPerVec;
  extern __shared__ __align__(16) uint4 buf[];               // the tile
  uint64_t* list = reinterpret_cast<uint64_t*>(buf + a.tile);  // a.cap entries
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t ubuf[32];
  __shared__ float fbuf[2][kWarps];
  __shared__ uint16_t hits[kHits];  // vectors of the tile with something at the bound
  __shared__ uint32_t n_list, n_hits;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t buf_at = (uint32_t)__cvta_generic_to_shared(buf) + tid * 16;

  // starts the copy of vector t0 + i of a row
  auto fetch = [&](const RowView<DT>& view, int64_t t0, int u) {
    const int i = u * kThreads + tid;
    if (i >= a.tile || t0 + i >= view.vectors()) return;
    if (view.whole(t0 + i)) copy_async(buf_at + u * kThreads * 16, view.p + view.first_of(t0 + i));
    else buf[i] = view.load(t0 + i);
  };
  int64_t row = blockIdx.x;
  if (row < a.rows) {
    const RowView<DT> view(a.x, row * a.stride, a.V);
    for (int u = 0; u < kVecs; u++) fetch(view, 0, u);
  }
  for (; row < a.rows; row += gridDim.x) {
    const RowView<DT> view(a.x, row * a.stride, a.V);
    const int64_t nv = view.vectors();
    uint64_t thr = 0;  // composites have to exceed it
    float m = neg_inf(), s = 0.0f;
    uint4 mx = neg_inf_vec<DT>();
    int n = 0;
    if (tid == 0) n_list = 0;
    for (int64_t t0 = 0; t0 < nv; t0 += a.tile) {
      const int here = (int)min((int64_t)a.tile, nv - t0);
      // where the copies of the pass below go on: the next tile or row
      const bool last = t0 + a.tile >= nv;
      const int64_t row2 = last ? row + gridDim.x : row;
      const RowView<DT> view2(a.x, (row2 < a.rows ? row2 : row) * a.stride, a.V);
      const int64_t t2 = last ? 0 : t0 + a.tile;
      const int64_t nv2 = row2 < a.rows ? view2.vectors() - t2 : 0;
      const int here2 = (int)min((int64_t)a.tile, nv2);
      const T* p2 = view2.p + view2.first_of(t2);
      const int lo2 = t2 == 0 && view2.shift ? 1 : 0;
      const int hi2 = here2 - (here2 > 0 && !view2.whole(t2 + here2 - 1) ? 1 : 0);

      // the groups' largest, and with them the thread's
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      if (tid == 0) n_hits = 0;
      copy_wait();
#pragma unroll 4
      for (int i = tid; i < here; i += kThreads) mx = max_vec<DT>(mx, buf[i]);
      float gmax[EPV], m2;
      E::unpack(mx, gmax);
#pragma unroll
      for (int g = GROUPS; g < EPV; g++) gmax[g % GROUPS] = fmaxf(gmax[g % GROUPS], gmax[g]);
      m2 = gmax[0];
      float low = gmax[0] > neg_inf() ? gmax[0] : INFINITY;
#pragma unroll
      for (int g = 1; g < GROUPS; g++) {
        m2 = fmaxf(m2, gmax[g]);
        low = fminf(low, gmax[g] > neg_inf() ? gmax[g] : INFINITY);
      }
      s *= ex2((shift_of(m) - shift_of(m2)) * a.c);
      m = m2;
      // the range of the groups' largest: finite ones
      float high = m < INFINITY ? m : 3.0e38f;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        low = fminf(low, __shfl_xor_sync(kFull, low, o));
        high = fmaxf(high, __shfl_xor_sync(kFull, high, o));
      }
      if (lane == 0) {
        fbuf[0][wid] = low;
        fbuf[1][wid] = high;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarps; i++) {
        low = fminf(low, fbuf[0][i]);
        high = fmaxf(high, fbuf[1][i]);
      }
      const float scale = high > low ? (float)kBins * 0.999f / (high - low) : 0.0f;
#pragma unroll
      for (int g = 0; g < GROUPS; g++)
        if (gmax[g] > neg_inf()) {
          const int b = min((int)((fminf(gmax[g], high) - low) * scale), kBins - 1);
          atomicAdd(&hist[b], 1u);
        }
      __syncthreads();
      // the last bin that has k of them in it and above (every warp for itself)
      float bound = neg_inf();
      {
        constexpr int per = kBins / 32;  // lane l: bins from the top, l * per and on
        uint32_t h[per], sum = 0;
#pragma unroll
        for (int j = 0; j < per; j++) {
          h[j] = hist[kBins - 1 - (lane * per + j)];
          sum += h[j];
        }
        const uint32_t inc = warp_incl_scan(sum, lane);
        const unsigned who = __ballot_sync(kFull, inc >= (uint32_t)a.k);
        if (who) {
          const int src = __ffs(who) - 1;
          uint32_t acc = inc - sum;
          int bin = 0;
#pragma unroll
          for (int j = 0; j < per; j++) {
            if (acc < (uint32_t)a.k) bin = kBins - 1 - (lane * per + j);
            acc += h[j];
          }
          bin = __shfl_sync(kFull, bin, src);
          // just under the bin: what fell into it is not below this, whatever
          // the roundings above
          if (bin > 0 && scale > 0.0f) bound = __fadd_rd(low, ((float)bin - 0.01f) / scale);
          else bound = low;
        }
      }
      const uint32_t bound2 = bound_of<DT>(bound);
      const float sh = shift_of(m);
      const pair_t c2 = pair(a.c, a.c), mc = pair(-sh * a.c, -sh * a.c);
      pair_t sum = pair(0.0f, 0.0f);
      auto take = [&](const uint4 r, int i) {
        float x[EPV];
        E::unpack(r, x);
#pragma unroll
        for (int j = 0; j < EPV; j += 2) sum = add2(sum, ex2_2(fma2(pair(x[j], x[j + 1]), c2, mc)));
        if (!all_below<DT>(r, bound2)) {
          const uint32_t at = atomicAdd(&n_hits, 1u);
          if (at < (uint32_t)kHits) hits[at] = (uint16_t)i;
        }
      };
#pragma unroll 1
      for (int u0 = 0; u0 < kVecs; u0 += kBlk) {
        if (u0 * kThreads >= here && u0 * kThreads >= here2) break;
        uint4 r[kBlk];
#pragma unroll
        for (int u = 0; u < kBlk; u++) {
          const int i = (u0 + u) * kThreads + tid;
          r[u] = i < here ? buf[i] : neg_inf_vec<DT>();
          if (i >= lo2 && i < hi2) copy_async(buf_at + (u0 + u) * kThreads * 16, p2 + (int64_t)i * EPV);
        }
#pragma unroll
        for (int u = 0; u < kBlk; u++)
          if ((u0 + u) * kThreads + wid * 32 < here) take(r[u], (u0 + u) * kThreads + tid);
      }
      s += sum.x + sum.y;
      // the ragged vectors of the next tile
      if (lo2 && tid == 0 && here2 > 0) buf[0] = view2.load(t2);
      if (hi2 < here2 && here2 > lo2 && (here2 - 1) % kThreads == tid) buf[here2 - 1] = view2.load(t2 + here2 - 1);
      __syncthreads();
      // the elements of the vectors that have something at the bound, read again
      // (from L2) and spread over the threads
      const int n_hit = (int)n_hits;
      if (n_hit <= kHits) {
        for (int q = tid; q < n_hit * EPV; q += kThreads) {
          const int64_t e = view.first_of(t0 + hits[q / EPV]) + q % EPV;
          if (e < 0 || e >= view.n) continue;
          const float x = E::load(view.p + e);
          const uint64_t v = (uint64_t)order_key(x) << 32 | (uint32_t)~(uint32_t)e;
          if (!(x < bound) && v > thr) {
            const uint32_t at = atomicAdd(&n_list, 1u);
            if (at < (uint32_t)a.cap) list[at] = v;
          }
        }
        __syncthreads();
        if (n_list <= (uint32_t)a.cap) {
          n = (int)n_list;
          continue;
        }
      }
      // too many: cut the list to the k best of before, then take the tile's own
      // k best above them, found bit by bit over a second read of it
      sort_list(list, n);
      if (n >= a.k) {
        n = a.k;
        thr = list[n - 1];
      }
      auto each = [&](auto f) {
#pragma unroll 1
        for (int i = tid; i < here; i += kThreads) {
          float x[EPV];
          E::unpack(view.load(t0 + i), x);
          const int64_t e0 = view.first_of(t0 + i);
#pragma unroll
          for (int j = 0; j < EPV; j++)
            if (e0 + j >= 0 && e0 + j < view.n) {
              const uint64_t v = (uint64_t)order_key(x[j]) << 32 | (uint32_t)~(uint32_t)(e0 + j);
              if (v > thr) f(v);
            }
        }
      };
      uint64_t cut = 0;
      for (int b = 63; b >= 0; b--) {
        const uint64_t t = cut | (1ull << b);
        uint32_t c = 0;
        each([&](uint64_t v) { c += v >= t; });
        c = cta_sum(c, ubuf);
        if (c >= (uint32_t)a.k) {
          cut = t;
          if (n + (int)c <= a.cap) break;
        }
      }
      if (tid == 0) n_list = n;
      __syncthreads();
      each([&](uint64_t v) {
        if (v >= cut) list[atomicAdd(&n_list, 1u)] = v;
      });
      __syncthreads();
      n = (int)n_list;
    }
    // in order
    if (n <= kCountSort) {
      uint64_t v = 0;
      int above = 0;
      if (tid < n) {
        v = list[tid];
#pragma unroll 4
        for (int i = 0; i < n; i++) above += list[i] > v;
      }
      __syncthreads();
      if (tid < n) list[above] = v;
      __syncthreads();
    } else {
      sort_list(list, n);
    }
    for (int i = tid; i < a.k; i += kThreads) {
      const int32_t e = (int32_t)~(uint32_t)list[i];
      a.idx[row * a.k + i] = e;
      if (a.vals) static_cast<T*>(a.vals)[row * a.k + i] = view.p[e];
    }
    if (a.lse) {
      const float M = cta_max(m, reinterpret_cast<float*>(ubuf)), sh = shift_of(M);
      const float S = cta_sum(s * ex2((shift_of(m) - sh) * a.c), reinterpret_cast<float*>(ubuf));
      if (tid == 0) a.lse[row] = sh / a.tau + logf(S);
    }
    __syncthreads();
  }
}

template <int DT, int GROUPS>
cudaError_t launch(TopkArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};  // the shared-memory opt-in is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(topk_rows<DT, GROUPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kTile * 16 + 4 * kMaxK * 8);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  constexpr int EPV = Elem<DT>::kPerVec;
  // tiles of one size, the last one a little shorter
  const int64_t nv = (a.V + 2 * EPV - 2) / EPV;
  const int64_t tiles = (nv + kTile - 1) / kTile;
  a.tile = (int)((nv + tiles - 1) / tiles);
  a.cap = 1024;
  while (a.cap < 3 * a.k) a.cap *= 2;
  const int64_t slots = (int64_t)num_sms() * 3;
  const int64_t rounds = (a.rows + slots - 1) / slots;
  const unsigned grid = (unsigned)((a.rows + rounds - 1) / rounds);
  topk_rows<DT, GROUPS><<<grid, kThreads, (size_t)a.tile * 16 + (size_t)a.cap * 8, s>>>(a);
  return cudaGetLastError();
}

// Groups: at least 4 k of them while a thread has that many places.
template <int DT>
cudaError_t launch_dt(TopkArgs& a, cudaStream_t s) {
  if (4 * a.k <= kThreads) return launch<DT, 1>(a, s);
  if (4 * a.k <= 2 * kThreads) return launch<DT, 2>(a, s);
  if (DT == SCAPE_F32 || 4 * a.k <= 4 * kThreads) return launch<DT, 4>(a, s);
  return launch<DT, Elem<DT>::kPerVec>(a, s);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SCAPE_BF16  ? launch_dt<SCAPE_BF16>(a, s)
                        : dtype == SCAPE_F16 ? launch_dt<SCAPE_F16>(a, s)
                                             : launch_dt<SCAPE_F32>(a, s);
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "topk_rows: %s", cudaGetErrorString(e));
}
