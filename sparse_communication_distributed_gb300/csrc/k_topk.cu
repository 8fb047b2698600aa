// The k largest logits of every row, in order, and the row's log-sum-exp: what
// a teacher leaves behind for distillation.
//
// Candidates are ranked by the unique composite key << 32 | ~index (order_key
// of objective.cuh), so that equal logits go to the lower index.  A CTA takes a
// row in tiles of up to 64 KB of shared memory (97 KB in the shape for long rows);
// each thread works on vectors that it copied itself.  One pass over a tile keeps, for each of G groups of
// elements (a group is one place or a few of the vectors that a thread sees),
// the group's largest element so far.  At least k elements reach the k-th
// largest of these G, so nothing below it is among the row's k best; a histogram
// of the G over their range gives a bound just under it.  A second pass notes the
// vectors that reach the bound -- for logits in no special order k (1 + k / 2G) of
// a first tile, a t-th part of that of the t-th tile -- and sums the exponentials.
// In the end the elements of the vectors noted that reach the last bound are
// listed, and ranked by counting what is above each; a list longer than the CTA
// has threads, or a part of a row, is sorted.  Where too much reaches the bound (many equal logits, few
// above -inf, adverse orders), the tile is read again and its own k-th best
// composite is found bit by bit.
//
// Few rows: a cluster of CTAs takes a row, each a part of it; the parts' k best
// go to the first CTA's shared memory and are sorted once more.
//
// Each logit is read once from HBM, which alone would take 61 us for 4096 x
// 50257 bf16; the kernel takes 116 us there (k 64, 52 % of the copy bandwidth) and
// 163 us for 1024 x 131072 fp32 (k 256, 49 %).  Issue is active 58 % of the time
// and DRAM busy 39 % (2048 rows): a row costs 21 thousand warp instructions, 74 us
// for 4096 rows at the full issue rate, so the instructions bound it before the
// bytes.  Half of them are in the two passes, the others in the phases of a tile and
// the ranking, which compares each entry of the list with each other; the phases
// (maxima, histogram, sums, ranking) wait for one another, which the other CTAs of
// the SM fill only in part.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "objective.cuh"
#include "scape_kernels.cuh"

#define SCAPE_API extern "C" __attribute__((visibility("default")))

namespace scape {
namespace {

// Threads of a CTA and CTAs of an SM: for rows of up to four tiles, for longer
// ones (1024 x 131072 fp32, k 256: 163 us against 180 with nine smaller tiles; at
// three, 4000 x 32000 fp32, 144 against 130), and for short ones.
template <int NT_, int CTAS_>
struct Shape {
  static constexpr int NT = NT_, CTAS = CTAS_;
  static constexpr int kSmem = (228 / CTAS_ - 3) * 1024;  // bytes of a CTA's tile, list and hits
};
using Wide = Shape<256, 3>;
using Large = Shape<384, 2>;
using Narrow = Shape<128, 7>;
constexpr int kNarrowVecs = 1024;  // rows up to this many vectors are short
constexpr int kBlk = 2;            // vectors a thread handles at a time
constexpr int kMaxK = 1024;
constexpr int kBins = 256;
constexpr int kMaxCluster = 8;

struct TopkArgs {
  const void* x;
  int64_t rows, V, stride;
  int k;
  int cap;          // list entries; k of an earlier tile and k new ones always fit
  int tile;         // vectors of a tile
  int list_at;      // where the list begins, in vectors
  int hits;         // vectors that can be noted
  bool keep;        // whether they are kept, or read again
  int cluster;      // CTAs of a row
  int part;         // vectors of each one's part
  float tau, c;     // temperature, log2(e) / temperature
  int32_t* idx;
  void* vals;
  float* lse;
};

// Sorts list[0..n) in descending order (bitonic, padded with 0).
template <int kThreads>
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

// Entries of list[0..n) above v; zeros follow up to a multiple of 4.
__device__ __forceinline__ int count_above(const uint64_t* list, int n, uint64_t v) {
  int above = 0;
#pragma unroll 2
  for (int i = 0; i < n; i += 4) {
    const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(list + i);
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(list + i + 2);
    above += (p.x > v) + (p.y > v) + (q.x > v) + (q.y > v);
  }
  return above;
}

// The shift of a row's sum: as shift_of, and 0 for a maximum of +inf, whose term
// and log-sum-exp are then +inf and not NaN.
__device__ __forceinline__ float sum_shift(float m) { return fabsf(m) < INFINITY ? m : 0.0f; }

// Order of floats as signed whole numbers, and back (its own inverse).
__device__ __forceinline__ int as_ordered(float f) {
  const int i = __float_as_int(f);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_ordered(int i) {
  return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF));
}

// GROUPS: groups of a thread (1, 2, 4 or 8 for 16-bit elements, up to 4 else).
template <int DT, int GROUPS, class SH>
__global__ __launch_bounds__(SH::NT, SH::CTAS) void topk_rows(const TopkArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int EPV = E::kPerVec, kThreads = SH::NT, kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint4 buf[];                 // the tile
  uint64_t* list = reinterpret_cast<uint64_t*>(buf + a.list_at);  // a.cap entries
  // vectors of the row with something at the bound: a.hits entries, and what they hold
  uint32_t* const hits = reinterpret_cast<uint32_t*>(list + a.cap);
  uint4* const kept = reinterpret_cast<uint4*>(hits + a.hits);
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ __align__(16) int range[2][kWarps];
  __shared__ uint32_t ubuf[32];
  // maximum and sum of each warp, and of each CTA of a row
  __shared__ float wsum[2][kWarps], parts[2][kMaxCluster];
  __shared__ uint32_t n_list, n_hits;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int V = (int)a.V;
  const uint32_t rank = a.cluster > 1 ? cluster_rank() : 0;
  const int first = (int)rank * a.part;  // vector of the row where this CTA starts
  const uint32_t buf_at = (uint32_t)__cvta_generic_to_shared(buf) + tid * 16;

  // A tile of a row: its first vector starts at p, coordinate e0 (< 0 where the
  // row starts inside it); "here" vectors, whole ones [lo, hi).
  struct Where {
    const T* p;
    int e0, here, lo, hi;
  };
  auto where = [&](const T* row_start, int t0) {
    Where w;
    w.e0 = t0 * EPV - (int)((reinterpret_cast<uintptr_t>(row_start) & 15u) / sizeof(T));
    w.p = row_start + w.e0;
    // elements from the tile's start; the last CTA of a row may have none
    const unsigned left = (unsigned)max((int64_t)V - w.e0, (int64_t)0);
    const unsigned most = (unsigned)min(a.tile, first + a.part - t0);
    w.here = (int)min(most, (left + EPV - 1) / EPV);
    w.lo = w.e0 < 0 ? 1 : 0;
    w.hi = (int)min(most, left / EPV);
    return w;
  };
  // starts the copies of the whole vectors among kBlk of this thread's
  auto fetch = [&](const Where& w, int u0) {
    const T* p = w.p + (int64_t)(u0 * kThreads + tid) * EPV;
#pragma unroll
    for (int u = 0; u < kBlk; u++) {
      const int i = (u0 + u) * kThreads + tid;
      if (i >= w.lo && i < w.hi) copy_async(buf_at + (u0 + u) * kThreads * 16, p + u * kThreads * EPV);
    }
  };
  // one element by itself, -inf outside the row
  auto element = [&](const Where& w, int l) {
    const int e = w.e0 + l;
    return e >= 0 && e < V ? E::load(w.p + l) : neg_inf();
  };
  // ... and puts ragged ones together
  auto fetch_ragged = [&](const Where& w) {
    auto one = [&](int i) {
      float f[EPV];
#pragma unroll
      for (int j = 0; j < EPV; j++) f[j] = element(w, i * EPV + j);
      buf[i] = E::pack(f);
    };
    if (w.lo && tid == 0) one(0);
    if (w.here > w.hi && w.here > w.lo && (w.here - 1) % kThreads == tid) one(w.here - 1);
  };

  const int64_t step = gridDim.x / (unsigned)a.cluster;
  int64_t row = blockIdx.x / (unsigned)a.cluster;
  const T* row_start = static_cast<const T*>(a.x) + row * a.stride;
  Where next = where(row_start, first);
  if (row < a.rows) {
    for (int u0 = 0; u0 * kThreads < next.hi; u0 += kBlk) fetch(next, u0);
    fetch_ragged(next);
  }
  for (; row < a.rows; row += step) {
    const T* const start = row_start;
    const int shift_e = (int)((reinterpret_cast<uintptr_t>(start) & 15u) / sizeof(T));
    row_start += step * a.stride;
    uint64_t thr = 0;  // composites have to exceed it
    float m = neg_inf(), s = 0.0f;
    uint4 mx = neg_inf_vec<DT>();
    int n = 0, before = 0;  // entries of the list, hits of the tiles before
    if (tid == 0) n_list = n_hits = 0;
    // an element's composite, if it is one of the row's
    auto composite = [&](int e, float x) { return (uint64_t)order_key(x) << 32 | (uint32_t)~(uint32_t)e; };
    // Takes the k best among what each(f) calls f for, and the list, into the
    // list: it is cut to its k best, and those above the last of them are found
    // bit by bit.
    auto select = [&](auto each) {
      sort_list<kThreads>(list, n);
      if (n >= a.k) {
        n = a.k;
        thr = list[n - 1];
      }
      auto above = [&](auto f) {
        each([&](int e) {
          if (e < 0 || e >= V) return;
          const uint64_t v = composite(e, E::load(start + e));
          if (v > thr) f(v);
        });
      };
      uint64_t cut = 0;
      for (int b = 63; b >= 0; b--) {
        const uint64_t t = cut | (1ull << b);
        uint32_t c = 0;
        above([&](uint64_t v) { c += v >= t; });
        c = cta_sum(c, ubuf);
        if (c >= (uint32_t)a.k) {
          cut = t;
          if (n + (int)c <= a.cap) break;
        }
      }
      if (tid == 0) n_list = n;
      __syncthreads();
      above([&](uint64_t v) {
        if (v >= cut) list[atomicAdd(&n_list, 1u)] = v;
      });
      __syncthreads();
      n = (int)n_list;
    };
    // Lists the elements of the first h hits that reach the bound, spread over the
    // threads; if they are not kept, they are read again, from L2 mostly.
    auto flush = [&](int h, float bound) {
      auto each = [&](auto f) {
        for (int q = tid; q < h * EPV; q += kThreads) f((int)hits[q / EPV] * EPV + q % EPV - shift_e, q);
      };
      each([&](int e, int q) {
        if (e < 0 || e >= V) return;
        const float x = a.keep ? E::load(reinterpret_cast<const T*>(kept) + q) : E::load(start + e);
        const uint64_t v = composite(e, x);
        if (!(x < bound) && v > thr) {
          const uint32_t at = atomicAdd(&n_list, 1u);
          if (at < (uint32_t)a.cap) list[at] = v;
        }
      });
      __syncthreads();
      if (n_list <= (uint32_t)a.cap) n = (int)n_list;
      else select([&](auto f) { each([&](int e, int) { f(e); }); });
    };
    for (int t0 = first;; t0 += a.tile) {
      const Where now = next;
      // where the copies of the listing pass go on: the next tile or row
      const bool last = t0 + a.tile >= first + a.part || (int64_t)now.e0 + now.here * EPV >= V;
      next = where(last ? row_start : start, last ? first : t0 + a.tile);
      if (last && row + step >= a.rows) next.here = next.lo = next.hi = 0;
      const int here = now.here;

      // the groups' largest, and with them the thread's
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      copy_wait();
#pragma unroll 4
      for (int i = tid; i < here; i += kThreads) mx = max_vec<DT>(mx, buf[i]);
      float gmax[EPV];
      E::unpack(mx, gmax);
#pragma unroll
      for (int g = GROUPS; g < EPV; g++) gmax[g % GROUPS] = fmaxf(gmax[g % GROUPS], gmax[g]);
      float m2 = gmax[0], low = gmax[0] > neg_inf() ? gmax[0] : INFINITY;
#pragma unroll
      for (int g = 1; g < GROUPS; g++) {
        m2 = fmaxf(m2, gmax[g]);
        low = fminf(low, gmax[g] > neg_inf() ? gmax[g] : INFINITY);
      }
      s *= ex2((m - sum_shift(m2)) * a.c);
      m = m2;
      // the range of the groups' largest: finite ones
      int ihigh = __reduce_max_sync(kFull, as_ordered(fminf(m, 3.0e38f)));
      int ilow = __reduce_min_sync(kFull, as_ordered(low));
      if (lane == 0) {
        range[0][wid] = ilow;
        range[1][wid] = ihigh;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarps; i += 4) {
        const int4 l = *reinterpret_cast<const int4*>(&range[0][i]);
        const int4 h = *reinterpret_cast<const int4*>(&range[1][i]);
        ilow = min(min(min(l.x, l.y), min(l.z, l.w)), ilow);
        ihigh = max(max(max(h.x, h.y), max(h.z, h.w)), ihigh);
      }
      low = from_ordered(ilow);
      const float high = from_ordered(ihigh);
      const float scale = high > low ? (float)kBins * 0.999f / (high - low) : 0.0f;
#pragma unroll
      for (int g = 0; g < GROUPS; g++)
        if (gmax[g] > neg_inf()) {
          const int b = min((int)((fminf(gmax[g], high) - low) * scale), kBins - 1);
          atomicAdd(&hist[b], 1u);
        }
      __syncthreads();
      // the last bin that has k of them in it and above (every warp for itself);
      // lane l has the bins from the top, l * per and on
      float bound = neg_inf();
      {
        constexpr int per = kBins / 32;
        uint32_t h[per], sum = 0;
#pragma unroll
        for (int j = 0; j < per; j += 4) {
          const uint4 q = *reinterpret_cast<const uint4*>(&hist[kBins - (lane * per + j) - 4]);
          h[j] = q.w; h[j + 1] = q.z; h[j + 2] = q.y; h[j + 3] = q.x;
        }
#pragma unroll
        for (int j = 0; j < per; j++) sum += h[j];
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
      const float sh = sum_shift(m);
      const Shift by(sh, a.c);  // (this thread's own maximum, far below the row's where all it has is masked)
      const pair_t c2 = pair(by.c, by.c), mc = pair(-by.k, -by.k);
      pair_t sum = pair(0.0f, 0.0f);
      auto take = [&](const uint4 r, int i, bool in) {
        float x[EPV];
        E::unpack(r, x);
#pragma unroll
        for (int j = 0; j < EPV; j += 2) sum = add2(sum, ex2_2(fma2(pair(x[j], x[j + 1]), c2, mc)));
        if (in && !all_below<DT>(r, bound2)) {
          const uint32_t at = atomicAdd(&n_hits, 1u);
          if (at < (uint32_t)a.hits) {
            hits[at] = (uint32_t)(t0 + i);
            if (a.keep) kept[at] = r;
          }
        }
      };
      // whole blocks of vectors, then the rest one by one
      int u0 = 0;
#pragma unroll 1
      for (; (u0 + kBlk) * kThreads <= here; u0 += kBlk) {
        uint4 r[kBlk];
#pragma unroll
        for (int u = 0; u < kBlk; u++) r[u] = buf[(u0 + u) * kThreads + tid];
        fetch(next, u0);
#pragma unroll
        for (int u = 0; u < kBlk; u++) take(r[u], (u0 + u) * kThreads + tid, true);
      }
#pragma unroll 1
      for (int u = u0; u * kThreads + wid * 32 < here; u++) {
        const int i = u * kThreads + tid;
        // (what a lane has beyond the tile counts for the sums alone: the vector there
        // is the next tile's or part's, and a bound of -inf would note it twice)
        take(i < here ? buf[i] : neg_inf_vec<DT>(), i, i < here);
      }
      for (; u0 * kThreads < next.hi; u0 += kBlk) fetch(next, u0);
      s += (sum.x + sum.y) * by.fix(sh);
      fetch_ragged(next);
      auto all_of_tile = [&](auto f) {
#pragma unroll 1
        for (int l = tid; l < here * EPV; l += kThreads) f(now.e0 + l);
      };
      __syncthreads();
      const int noted = (int)n_hits;
      if (noted > a.hits / 2 && !last) {
        // room for the tiles to come; too many in this tile: it goes another way
        flush(noted <= a.hits ? noted : before, bound);
        if (noted > a.hits) select(all_of_tile);
        __syncthreads();
        if (tid == 0) n_hits = 0;
        before = 0;
        continue;
      }
      if (noted > a.hits) {
        flush(before, bound);
        select(all_of_tile);
        break;
      }
      before = noted;
      if (last) {
        flush(before, bound);
        break;
      }
    }
    // each warp's maximum and sum of exponentials
    float M = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    float S = s * ex2((m - sum_shift(M)) * a.c);
#pragma unroll
    for (int o = 16; o; o >>= 1) S += __shfl_xor_sync(kFull, S, o);
    if (lane == 0) {
      wsum[0][wid] = M;
      wsum[1][wid] = S;
    }
    auto total = [&](const float* ms, const float* ss, int count) {  // of the first lanes' parts
      const float pm = lane < count ? ms[lane] : neg_inf(), ps = lane < count ? ss[lane] : 0.0f;
      M = pm;
#pragma unroll
      for (int o = 8; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
      S = ps * ex2((pm - sum_shift(M)) * a.c);
#pragma unroll
      for (int o = 8; o; o >>= 1) S += __shfl_xor_sync(kFull, S, o);
    };
    auto write = [&](int at, uint64_t v) {
      const int32_t e = (int32_t)~(uint32_t)v;
      a.idx[row * a.k + at] = e;
      if (a.vals) {  // only zeros and NaN have several logits to a key
        const float x = value_of_key((uint32_t)(v >> 32));
        static_cast<T*>(a.vals)[row * a.k + at] = x == 0.0f || x != x ? start[e] : E::make(x);
      }
    };
    auto write_lse = [&]() {
      if (a.lse && tid == 0) a.lse[row] = sum_shift(M) / a.tau + logf(S);
    };
    if (a.cluster == 1 && n <= kThreads) {  // by counting what is above each entry
      for (int i = n + tid; i < ((n + 3) & ~3); i += kThreads) list[i] = 0;
      __syncthreads();
      if (tid < n) {
        const uint64_t v = list[tid];
        const int above = count_above(list, n, v);
        if (above < a.k) write(above, v);
      }
      if (wid == 0) total(wsum[0], wsum[1], kWarps);
      write_lse();
    } else {
      sort_list<kThreads>(list, n);
      if (wid == 0) total(wsum[0], wsum[1], kWarps);
      if (a.cluster > 1) {  // (a single row for each cluster: the tile's space is free)
        uint64_t* all = reinterpret_cast<uint64_t*>(buf);  // k entries of each CTA
        cluster_arrive();
        cluster_wait();
        for (int i = tid; i < a.k; i += kThreads) put_remote(all + rank * a.k + i, 0, i < n ? list[i] : 0);
        if (tid == 0) {
          put_remote(&parts[0][rank], 0, M);
          put_remote(&parts[1][rank], 0, S);
        }
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        list = all;
        sort_list<kThreads>(list, a.cluster * a.k);
        if (wid == 0) total(parts[0], parts[1], a.cluster);
      }
      for (int i = tid; i < a.k; i += kThreads) write(i, list[i]);
      write_lse();
    }
    __syncthreads();
  }
}

template <int DT, int GROUPS, class SH>
cudaError_t launch(TopkArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};  // the shared-memory opt-in is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(topk_rows<DT, GROUPS, SH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SH::kSmem + kMaxCluster * kMaxK * 8);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  // tiles of one size that fit beside the list, the last one a little shorter
  constexpr int EPV = Elem<DT>::kPerVec;
  a.cap = 512;
  while (a.cap < 3 * a.k) a.cap *= 2;
  const bool whole = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.stride % EPV == 0;
  const int64_t nv = (a.V + (whole ? 0 : EPV - 1) + EPV - 1) / EPV;
  a.cluster = 1;  // few rows: more CTAs for each, down to two vectors a thread
  while (a.cluster < kMaxCluster && a.rows * a.cluster <= num_sms() && nv > 4 * SH::NT * a.cluster)
    a.cluster *= 2;
  a.part = (int)((nv + a.cluster - 1) / a.cluster);
  // noted vectors are kept where a quarter of the memory holds them and the list
  // (4096 x 50257 bf16, k 64: 120 us against 125; k 256 in large tiles, 1024 x
  // 131072 fp32: 169 against 166)
  a.hits = std::max(256, (4 * a.k + 3) & ~3);
  a.keep = a.cap * 8 + a.hits * 20 <= SH::kSmem / 4;
  if (!a.keep) a.hits = std::max(1024, 6 * a.k);
  const int hit_bytes = a.hits * (a.keep ? 20 : 4);
  const int64_t most = (SH::kSmem - a.cap * 8 - hit_bytes) / 16;
  const int64_t tiles = (a.part + most - 1) / most;
  a.tile = (int)((a.part + tiles - 1) / tiles);
  size_t bytes = (size_t)a.tile * 16;
  if (a.cluster > 1) {  // the parts' entries, and what their sort pads
    size_t n = 1;
    while (n < (size_t)a.cluster * a.k) n *= 2;
    bytes = std::max(bytes, n * 8);
  }
  a.list_at = (int)(bytes + 15) / 16;
  const int64_t slots = (int64_t)num_sms() * SH::CTAS;
  const int64_t rounds = (a.rows * a.cluster + slots - 1) / slots;
  const int64_t clusters = (a.rows + rounds - 1) / rounds;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * a.cluster));
  cfg.blockDim = dim3(SH::NT);
  cfg.dynamicSmemBytes = (size_t)a.list_at * 16 + (size_t)a.cap * 8 + (size_t)hit_bytes;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)a.cluster;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, topk_rows<DT, GROUPS, SH>, a);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

// Groups: at least 4 k of them while a thread has that many places.
template <int DT, class SH>
cudaError_t launch_groups(TopkArgs& a, cudaStream_t s) {
  if (4 * a.k <= SH::NT) return launch<DT, 1, SH>(a, s);
  if (4 * a.k <= 2 * SH::NT) return launch<DT, 2, SH>(a, s);
  if (DT == SCAPE_F32 || 4 * a.k <= 4 * SH::NT) return launch<DT, 4, SH>(a, s);
  return launch<DT, Elem<DT>::kPerVec, SH>(a, s);
}

template <int DT>
cudaError_t launch_dt(TopkArgs& a, cudaStream_t s) {
  // (a narrow CTA's list holds 3 k entries beside its row for k up to this)
  if (a.V <= (kNarrowVecs - 1) * Elem<DT>::kPerVec && a.k <= 256) return launch_groups<DT, Narrow>(a, s);
  const bool longer = a.V > 4 * (Wide::kSmem - 3 * 4096) / 16 * Elem<DT>::kPerVec;
  return longer ? launch_groups<DT, Large>(a, s) : launch_groups<DT, Wide>(a, s);
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
