// Expert routing: top-k experts of every token, their weights, how many
// choices every expert of every group of tokens got, the balance loss and the z
// loss; and the gradient of the logits.
//
// Forward.  A token's logits lie across L lanes of a warp, so that a warp works
// on 32 / L tokens at once (L = 8 for 33 to 256 experts).  The choice goes the
// way of the top logits: of each of at least 32 groups of experts (or of each
// expert) the largest logit is known, the k-th largest of those is a bound that
// at least k experts reach, and only the few that do are put into a list and
// ranked by comparing each with each.  Rows with too many of them (many equal
// logits) are done one choice after the other.
//
// The tokens are cut into chunks, one CTA each; within a chunk the CTA goes group
// by group and leaves, for every group that the chunk touches, the sums of p and
// the counts over its tokens in a slot of the workspace.  Chunk i and group g
// use slot i + g: along the tokens either i or g moves on, so no two pairs share
// a slot and a group's slots are adjacent.  A second kernel adds a group's slots
// up in order, so the sums do not depend on the schedule.
//
// Backward.  With d_e = dB / G' * E c_ge / (k T_g^2) of the token's group,
//   d x_j = p_j (d_j - sum_e p_e d_e) + (2 dZ / T) lse p_j + (weights' part),
// where the weights' part is w_i (dw_i - sum w dw) at the chosen experts if
// renormalised, else p_j (dw_j [chosen] - sum w dw).
//
// Instructions are the bound, not bytes.  Forward, 131072 x 256 fp32 with k 8: 60
// us in all, 35 % of the copy bandwidth, bf16 60 us (18 %).  A token of 256 experts
// costs 235 warp instructions (three quarters for the bound, list, ranks and output
// of the four tokens of a warp, whatever their width), and 16 warps an SM, as the
// logits, the sums over the tokens and the next token's logits fill 128 registers,
// issue half of the time.  They do not all fit: above 128 experts the forward spills
// up to 8 bytes a thread in fp32 and 76 to 108 in 16 bits, the backward 8 to 180 in 16 bits
// and 124 to 392 in fp32.  A ragged batch of 16384 x 64 is bound by latency: 15.5 us
// in a graph, two rounds of tokens and a second kernel's chain of sums.  Backward,
// 65536 x 128 bf16 with k 8 and 32 groups: 16 us, hardly more than the call costs the
// host; 524288 tokens 82 us, 55 % of the copy bandwidth; 65536 x 256 bf16 23 us, fp32
// 41 us (49 %).
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
constexpr int kMaxK = 32;
constexpr int kMaxExperts = 1024;

struct RouteArgs {
  const void* x;
  int64_t T, stride;
  int E, k, renorm;
  bool single;     // one chunk and one group
  bool vec, gvec;  // rows of the logits, of the gradient in whole 16-byte vectors
  const int32_t* cu;
  int64_t G;
  const uint8_t* valid;
  int64_t chunk;  // tokens of a CTA
  // forward
  int32_t* idx;
  float* weights;
  float* part_p;       // slots x E: sums of p
  int32_t* part_c;     // slots x E: choices
  int32_t* part_n;     // slots: live tokens
  float* part_z;       // slots: sum of lse^2
  uint32_t* done;      // CTAs of the second kernel that have finished
  float* part_b;       // groups x column blocks of the second kernel
  float* group_z;      // groups: sum of lse^2
  int32_t* counts;
  int32_t* live;
  float* losses;
  // backward
  const int32_t* bidx;
  const int32_t* bcounts;
  const int32_t* blive;
  const float* dw;
  const float* dl;
  void* grad;
  int64_t gstride;
};

// Tokens [lo, hi) of group g, clamped to [0, T] whatever cu holds.
__device__ __forceinline__ int64_t bound_of(const RouteArgs& a, int64_t g) {
  if (!a.cu) return g <= 0 ? 0 : a.T;
  const int64_t v = a.cu[g];
  return v < 0 ? 0 : v > a.T ? a.T : v;
}

// First group whose end lies beyond token t (a.G if none), found by a whole
// warp for one t: 32 probes at a time.
__device__ __forceinline__ int64_t group_at(const RouteArgs& a, int64_t t) {
  if (!a.cu) return t < a.T ? 0 : 1;
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = a.G;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, probe = min(lo + (lane + 1) * step, hi) - 1;
    const unsigned beyond = __ballot_sync(kFull, bound_of(a, probe + 1) > t);
    if (!beyond) return hi;  // the last probe is hi - 1
    const int first = __ffs(beyond) - 1;
    hi = min(lo + (first + 1) * step, hi) - 1;
    lo += first * step;
    if (step == 1) return hi;
  }
  return lo;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int o = L >> 1; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
template <int L>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
  for (int o = L >> 1; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}

// How a token's experts lie in a warp: L lanes, VPL values each, in vectors of
// 16 bytes that follow each other over the lanes.  GPL groups of a lane's values
// for the bound.
template <int L_, int VPL_, int GPL_>
struct Lanes {
  static constexpr int L = L_, VPL = VPL_, GPL = GPL_, ROWS = 32 / L_;
  static constexpr int CAP = L_ * VPL_ < 48 ? L_ * VPL_ : 48;  // list entries of a token
  static_assert(CAP % 4 == 0, "the list is read in fours");
};

template <int DT, int L>
__device__ __forceinline__ int col_of(int sub, int j) {
  constexpr int N = Elem<DT>::kPerVec;
  return (j / N * L + sub) * N + j % N;
}

// A lane's logits of one token as they lie in memory, -inf beyond the experts.
// vec: rows on 16-byte boundaries and whole vectors.  The loads stay in L1, where
// the few logits looked up by expert are found again (131072 x 256 fp32: 82 -> 73
// us against loads that do not).
template <int DT, class LN>
struct RowRegs {
  static constexpr int N = Elem<DT>::kPerVec, VECS = LN::VPL / N;
  uint4 r[VECS];
  __device__ __forceinline__ void load(const typename Elem<DT>::T* p, int E, int sub, bool in, bool vec) {
    if (vec) {
      p += sub * N;
      E = in ? E - sub * N : 0;
#pragma unroll
      for (int v = 0; v < VECS; v++) {
        r[v] = neg_inf_vec<DT>();
        if (v * LN::L * N < E) r[v] = *reinterpret_cast<const uint4*>(p + v * LN::L * N);
      }
    } else {
#pragma unroll
      for (int v = 0; v < VECS; v++) {
        const int col = (v * LN::L + sub) * N;
        float f[N];
#pragma unroll
        for (int j = 0; j < N; j++) f[j] = in && col + j < E ? Elem<DT>::load(p + col + j) : neg_inf();
        r[v] = Elem<DT>::pack(f);
      }
    }
  }
  __device__ __forceinline__ void get(float (&x)[LN::VPL]) const {
#pragma unroll
    for (int v = 0; v < VECS; v++) {
      float f[N];
      Elem<DT>::unpack(r[v], f);
#pragma unroll
      for (int j = 0; j < N; j++) x[v * N + j] = f[j];
    }
  }
};

// A bound that at least k of a token's experts reach, from the largest logits of
// its L x GPL groups: the k-th largest of the lanes' two largest of them, i from
// the largest and k - i from the second largest.  Of 256 experts 9.4 reach it on
// average for k = 8, where 8.9 reach the k-th largest of all groups, which takes
// five times the instructions.  Where k is above 3 L / 2 the lanes' third ones
// count (17 against 14 for k = 12, 38 against 21 for k = 16), and it is that exact
// one.
template <class LN>
__device__ __forceinline__ float bound_for(float (&gm)[LN::GPL], int k, int lane, unsigned seg) {
  constexpr int L = LN::L, GPL = LN::GPL;
  if (k <= (GPL > 1 ? L + L / 2 : L)) {
    float top = neg_inf(), second = neg_inf();
#pragma unroll
    for (int j = 0; j < GPL; j++) {
      second = fmaxf(second, fminf(top, gm[j]));
      top = fmaxf(top, gm[j]);
    }
    // both in descending order over the lanes
#pragma unroll
    for (int size = 2; size <= L; size <<= 1)
#pragma unroll
      for (int d = size >> 1; d; d >>= 1) {
        const bool keep_max = ((lane & d) == 0) == ((lane & size) == 0 || size == L);
        const float t = __shfl_xor_sync(kFull, top, d);
        top = keep_max ? fmaxf(top, t) : fminf(top, t);
        if (GPL > 1) {
          const float u = __shfl_xor_sync(kFull, second, d);
          second = keep_max ? fmaxf(second, u) : fminf(second, u);
        }
      }
    if (GPL == 1) return __shfl_sync(kFull, top, k - 1, L);
    const int j = k - 2 - (lane & (L - 1));  // the last of the k - i second ones
    const float u = __shfl_sync(kFull, second, j & (L - 1), L);
    const float both = j < 0 ? top : fminf(top, u);
    return lanes_max<L>(j >= -1 && j < L ? both : neg_inf());
  }
  float bound = neg_inf();
  for (int i = 0; i < k; i++) {
    float h = gm[0];
#pragma unroll
    for (int j = 1; j < GPL; j++) h = fmaxf(h, gm[j]);
    bound = lanes_max<L>(h);
    // one of those that are equal to it is taken out
    const unsigned who = __ballot_sync(kFull, h == bound) & seg;
    bool mine = lane == __ffs(who) - 1;
#pragma unroll
    for (int j = 0; j < GPL; j++) {
      const bool hit = mine && gm[j] == bound;
      gm[j] = hit ? neg_inf() : gm[j];
      mine = mine && !hit;
    }
  }
  return bound;
}

template <int DT, class LN>
__global__ __launch_bounds__(kThreads, 2) void route_chunks(const RouteArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int L = LN::L, VPL = LN::VPL, GPL = LN::GPL, ROWS = LN::ROWS, CAP = LN::CAP;
  extern __shared__ __align__(16) unsigned char smem[];
  uint64_t* lists = reinterpret_cast<uint64_t*>(smem);  // kWarps x ROWS x CAP
  uint64_t* ranks = lists + kWarps * ROWS * CAP;                      // kWarps x ROWS x k
  float* sp = reinterpret_cast<float*>(ranks + kWarps * ROWS * a.k);  // kWarps x E
  int32_t* sc = reinterpret_cast<int32_t*>(sp + kWarps * a.E);        // E
  __shared__ float fbuf[32];
  __shared__ int32_t ibuf[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int sub = lane & (L - 1), slot = lane / L;
  const unsigned seg = (L == 32 ? kFull : ((1u << L) - 1u) << (slot * L));  // this token's lanes
  uint64_t* list = lists + (wid * ROWS + slot) * CAP;
  uint64_t* sorted = ranks + (wid * ROWS + slot) * a.k;
  uint32_t experts = 0;  // this lane's values that are experts, value j at bit VPL - 1 - j
#pragma unroll
  for (int j = 0; j < VPL; j++)
    if (col_of<DT, L>(sub, j) < a.E) experts |= 1u << (VPL - 1 - j);
  const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  if (blockIdx.x == 0 && tid == 0 && !a.single) *a.done = 0;
  grid_launch_dependents();  // the second kernel waits for this one on its own

  // pieces of the chunk: each group it touches, and tokens outside all groups
  int64_t at = t0, g = group_at(a, t0);
  while (at < t1) {
    int64_t end = t1;
    bool inside = false;
    if (g < a.G) {
      const int64_t lo = bound_of(a, g), hi = bound_of(a, g + 1);
      if (lo > at) end = min(lo, t1);
      else {
        end = min(hi, t1);
        inside = true;
      }
      if (end <= at) {  // an empty group, or bounds out of order
        g++;
        continue;
      }
    }
    pair_t acc[VPL / 2];
#pragma unroll
    for (int j = 0; j < VPL / 2; j++) acc[j] = pair(0.0f, 0.0f);
    float zsum = 0.0f;
    int32_t nlive = 0;
    for (int i = tid; i < a.E; i += kThreads) sc[i] = 0;
    __syncthreads();
    RowRegs<DT, LN> next;
    int64_t t = at + wid * ROWS + slot;
    next.load(static_cast<const T*>(a.x) + t * a.stride, a.E, sub, t < end, a.vec);
    for (int64_t r = at + wid * ROWS; r < end; r += kWarps * ROWS, t += kWarps * ROWS) {
      const bool in = t < end;
      const T* p_row = static_cast<const T*>(a.x) + t * a.stride;
      float x[VPL];
      next.get(x);
      next.load(p_row + kWarps * ROWS * a.stride, a.E, sub, t + kWarps * ROWS < end, a.vec);
      bool ok = in && inside && (!a.valid || a.valid[t] != 0);
      float gm[GPL];
#pragma unroll
      for (int j = 0; j < GPL; j++) gm[j] = x[j];
#pragma unroll
      for (int j = GPL; j < VPL; j++) gm[j % GPL] = fmaxf(gm[j % GPL], x[j]);
      float m = gm[0];
#pragma unroll
      for (int j = 1; j < GPL; j++) m = fmaxf(m, gm[j]);
      m = lanes_max<L>(m);
      const float sh = shift_of(m);

      float bound = bound_for<LN>(gm, a.k, lane, seg);
      if (bound == 0.0f) bound = -0.0f;  // -0 - (-0) = +0, as 0 - (-0)
      // the experts that reach it, from the sign of the difference (positive or
      // NaN where not below): value j at bit VPL - 1 - j
      uint32_t cand = 0;
#pragma unroll
      for (int j = 0; j < VPL; j += 2) {
        const pair_t d = add2(pair(x[j], x[j + 1]), pair(-bound, -bound));
        cand = __funnelshift_l(__float_as_uint(d.x), cand, 1);
        cand = __funnelshift_l(__float_as_uint(d.y), cand, 1);
      }
      cand = ~cand & experts;

      // p, and the sums
      const Shift by(sh, kLog2e);  // (all logits may be the type's lowest value)
      const pair_t c2 = pair(by.c, by.c), mc = pair(-by.k, -by.k);
      pair_t s2 = pair(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < VPL; j += 2) {
        const pair_t e = ex2_2(fma2(pair(x[j], x[j + 1]), c2, mc));
        s2 = add2(s2, e);
        x[j] = e.x;
        x[j + 1] = e.y;
      }
      const float s = lanes_sum<L>(s2.x + s2.y);
      const float inv = rcp(s);
      ok = ok && !(s == 0.0f);  // some logit above -inf
      const float lse = sh + logf(s);
      if (ok) {
#pragma unroll
        for (int j = 0; j < VPL / 2; j++)
          acc[j] = fma2(pair(x[2 * j], x[2 * j + 1]), pair(inv, inv), acc[j]);
        if (sub == 0) {
          zsum += lse * lse;
          nlive++;
        }
      } else {
        cand = 0;
      }

      // listed: column first, then the composite
      int incl = __popc(cand);
#pragma unroll
      for (int o = 1; o < L; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o, L);
        if (sub >= o) incl += y;
      }
      const int n = __shfl_sync(kFull, incl, L - 1, L);
      for (int at_ = incl - __popc(cand); cand; at_++) {
        const int j = VPL - __ffs(cand);
        cand &= cand - 1;
        if (at_ < CAP) list[at_] = (uint64_t)col_of<DT, L>(sub, j);
      }
      __syncwarp();
      if (__any_sync(kFull, n > CAP)) {
        // one choice after the other, all logits read again
        uint32_t key[VPL];
        const bool all = in && ok;
#pragma unroll
        for (int j = 0; j < VPL; j++) {
          const int col = col_of<DT, L>(sub, j);
          key[j] = all && col < a.E ? order_key(E::load(p_row + col)) : 0u;
        }
        for (int i = 0; i < a.k; i++) {
          uint64_t best = 0;
#pragma unroll
          for (int j = 0; j < VPL; j++) {
            const uint64_t v = (uint64_t)key[j] << 32 | (uint32_t)~col_of<DT, L>(sub, j);
            best = v > best && key[j] ? v : best;
          }
#pragma unroll
          for (int o = L >> 1; o; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(kFull, best, o);
            best = other > best ? other : best;
          }
          const int col = (int)~(uint32_t)best;
#pragma unroll
          for (int j = 0; j < VPL; j++)
            if (col_of<DT, L>(sub, j) == col) key[j] = 0;
          if (sub == 0) sorted[i] = best;
        }
      } else {
        // ranked: each entry counts those above it
        for (int i = sub; i < n; i += L) {
          const uint32_t col = (uint32_t)list[i];
          list[i] = (uint64_t)order_key(E::load(p_row + col)) << 32 | (uint32_t)~col;
        }
        const int n4 = (n + 3) & ~3;  // at most CAP, a multiple of 4
        for (int i = n + sub; i < n4; i += L) list[i] = 0;
        __syncwarp();
        for (int i = sub; i < n; i += 2 * L) {  // two of a lane at a time
          const bool two = i + L < n;
          const uint64_t v = list[i], w = two ? list[i + L] : 0;
          int above = 0, above2 = 0;
#pragma unroll 1
          for (int q = 0; q < n; q += 4) {  // in fours: below the end come zeros
            const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(list + q);
            const ulonglong2 t2 = *reinterpret_cast<const ulonglong2*>(list + q + 2);
            above += (u.x > v) + (u.y > v) + (t2.x > v) + (t2.y > v);
            above2 += (u.x > w) + (u.y > w) + (t2.x > w) + (t2.y > w);
          }
          if (above < a.k) sorted[above] = v;
          if (two && above2 < a.k) sorted[above2] = w;
        }
      }
      __syncwarp();
      float chosen = 0.0f;
      if (a.renorm && ok)
        for (int i = sub; i < a.k; i += L)
          chosen += by.term(value_of_key((uint32_t)(sorted[i] >> 32)));
      const float scale = a.renorm ? rcp(lanes_sum<L>(chosen)) : inv;
      if (in)
        for (int i = sub; i < a.k; i += L) {
          const uint64_t v = ok ? sorted[i] : 0;
          const int col = (int)~(uint32_t)v;  // -1 for v = 0
          a.idx[t * a.k + i] = col;
          a.weights[t * a.k + i] = ok ? by.term(value_of_key((uint32_t)(v >> 32))) * scale : 0.0f;
          if (ok) atomicAdd(&sc[col], 1);
        }
      __syncwarp();
    }
    if (inside) {  // the slot of this chunk and group
#pragma unroll
      for (int j = 0; j < VPL; j++) {
        float v = j % 2 ? acc[j / 2].y : acc[j / 2].x;
#pragma unroll
        for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(kFull, v, o);
        const int col = col_of<DT, L>(sub, j);
        if (slot == 0 && col < a.E) sp[wid * a.E + col] = v;
      }
      const float z = cta_sum(zsum, fbuf);
      const int32_t nl = cta_sum(nlive, ibuf);
      __syncthreads();
      const int64_t sl = blockIdx.x + g;
      float b = 0.0f;
      for (int i = tid; i < a.E; i += kThreads) {
        float p = 0.0f;
        for (int w = 0; w < kWarps; w++) p += sp[w * a.E + i];
        if (a.single) {
          a.counts[i] = sc[i];
          b += p * (float)sc[i];
        } else {
          a.part_p[sl * a.E + i] = p;
          a.part_c[sl * a.E + i] = sc[i];
        }
      }
      if (a.single) {  // one CTA has it all: no second kernel
        const float tg = (float)max(nl, 1);
        b = cta_sum(b, fbuf) * ((float)a.E / ((float)a.k * tg)) / tg;
        if (tid == 0) {
          a.live[0] = a.live[1] = nl;
          a.live[2] = nl > 0;
          a.losses[0] = b;
          a.losses[1] = z / tg;
        }
      } else if (tid == 0) {
        a.part_n[sl] = nl;
        a.part_z[sl] = z;
      }
    }
    __syncthreads();
    if (g < a.G && bound_of(a, g + 1) <= end) g++;
    at = end;
  }
}

// One CTA per group and block of 8 columns (a sector of the slots); 32 threads
// share a column's slots.  The last CTA to finish adds up what the groups
// contribute.
constexpr int kCols = 8;

__global__ __launch_bounds__(kThreads) void route_finish(const RouteArgs a) {
  __shared__ float fbuf[32], sp[kWarps][kCols];
  __shared__ int32_t ibuf[32], sc[kWarps][kCols];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int64_t g = blockIdx.x;
  const int nb = gridDim.y;
  const int64_t lo = bound_of(a, g), hi = bound_of(a, g + 1);
  const int64_t s0 = lo / a.chunk + g, s1 = hi > lo ? (hi - 1) / a.chunk + g + 1 : s0;
  grid_dependency_wait();
  const int col = blockIdx.y * kCols + (lane & 7);
  float p = 0.0f;
  int32_t c = 0;
  if (col < a.E) {
#pragma unroll 4
    for (int64_t s = s0 + tid / kCols; s < s1; s += kThreads / kCols) {
      p += a.part_p[s * a.E + col];
      c += a.part_c[s * a.E + col];
    }
  }
  int32_t n = 0;
  float zg = 0.0f;
  for (int64_t s = s0 + tid; s < s1; s += kThreads) {
    n += a.part_n[s];
    zg += a.part_z[s];
  }
  n = cta_sum(n, ibuf);
  zg = cta_sum(zg, fbuf);
#pragma unroll
  for (int o = 16; o >= kCols; o >>= 1) {
    p += __shfl_xor_sync(kFull, p, o);
    c += __shfl_xor_sync(kFull, c, o);
  }
  if (lane < kCols) {
    sp[wid][lane] = p;
    sc[wid][lane] = c;
  }
  __syncthreads();
  float b = 0.0f;
  if (tid < kCols && col < a.E) {
    p = 0.0f;
    c = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      p += sp[w][tid];
      c += sc[w][tid];
    }
    a.counts[g * a.E + col] = c;
    b = p * (float)c;
  }
  const float tg = (float)max(n, 1);
  const float bal = cta_sum(b, fbuf) * ((float)a.E / ((float)a.k * tg)) / tg;
  if (tid == 0) {
    a.part_b[g * nb + blockIdx.y] = bal;
    if (blockIdx.y == 0) {
      a.live[g] = n;
      a.group_z[g] = zg;
    }
    __threadfence();
    last = atomicAdd(a.done, 1u) == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float sum = 0.0f, z = 0.0f;
  int32_t total = 0, groups = 0;
  for (int64_t i = tid; i < a.G * nb; i += kThreads) sum += __ldcg(a.part_b + i);
  for (int64_t i = tid; i < a.G; i += kThreads) {
    const int32_t v = __ldcg(a.live + i);
    total += v;
    groups += v > 0;
    z += __ldcg(a.group_z + i);
  }
  sum = cta_sum(sum, fbuf);
  z = cta_sum(z, fbuf);
  total = cta_sum(total, ibuf);
  groups = cta_sum(groups, ibuf);
  if (tid == 0) {
    a.live[a.G] = total;
    a.live[a.G + 1] = groups;
    a.losses[0] = sum / (float)max(groups, 1);
    a.losses[1] = z / (float)max(total, 1);
  }
}

template <int DT, class LN>
__global__ __launch_bounds__(kThreads, 2) void route_grad(const RouteArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int L = LN::L, VPL = LN::VPL, ROWS = LN::ROWS, N = E::kPerVec;
  // choices of a lane at most (k <= 32, and k <= experts); loops over them end at k
  // (524288 x 128 bf16, k 8: 82 us, 91 without)
  constexpr int KPL = 32 / L < 8 ? 32 / L : 8;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int sub = lane & (L - 1), slot = lane / L;
  const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  constexpr int64_t kStep = kWarps * ROWS;
  int64_t t = t0 + wid * ROWS + slot;
  // a token's inputs: its logits and choices are loaded a round ahead, the
  // logits at the choices at the end of the round before
  RowRegs<DT, LN> next;
  int32_t next_id[KPL], next_first = -1;
  float next_dw[KPL], next_x[KPL];
  auto fetch = [&](int64_t u) {
    const bool in = u < t1;
    next.load(static_cast<const T*>(a.x) + u * a.stride, a.E, sub, in, a.vec);
    next_first = in ? a.bidx[u * a.k] : -1;  // tells whether the token is live
#pragma unroll
    for (int q = 0; q < KPL; q++) {
      if (q * L >= a.k) break;
      const int i = q * L + sub;
      next_id[q] = -1;
      next_dw[q] = 0.0f;
      if (in && a.dw && i < a.k) {
        next_id[q] = a.bidx[u * a.k + i];
        next_dw[q] = a.dw[u * a.k + i];
      }
    }
  };
  auto fetch_chosen = [&](int64_t u) {
#pragma unroll
    for (int q = 0; q < KPL; q++) {
      if (q * L >= a.k) break;
      next_x[q] = neg_inf();
      if (next_id[q] >= 0 && next_id[q] < a.E)
        next_x[q] = E::load(static_cast<const T*>(a.x) + u * a.stride + next_id[q]);
    }
  };
  fetch(t);
  const float dB = a.dl ? a.dl[0] : 0.0f, dZ = a.dl ? a.dl[1] : 0.0f;
  const float zc = 2.0f * dZ / (float)max(a.blive[a.G], 1);
  const float bc = dB / (float)max(a.blive[a.G + 1], 1) * ((float)a.E / (float)a.k);
  // this token's group: its end, and d of this lane's experts
  int64_t g = group_at(a, t0), g_end = t0;
  const int32_t* gc = nullptr;
  float coef = 0.0f, d[VPL];
#pragma unroll
  for (int j = 0; j < VPL; j++) d[j] = 0.0f;
  fetch_chosen(t);
  for (int64_t r = t0 + wid * ROWS; r < t1; r += kStep, t += kStep) {
    const bool in = t < t1, ok = in && next_first >= 0;
    float x[VPL], xc[KPL], dwc[KPL];
    int id[KPL];
    next.get(x);
#pragma unroll
    for (int q = 0; q < KPL; q++) {
      if (q * L >= a.k) break;
      id[q] = next_id[q];
      dwc[q] = next_dw[q];
      xc[q] = next_x[q];
    }
    fetch(t + kStep);
    if (in && t >= g_end) {
      while (g < a.G && bound_of(a, g + 1) <= t) g++;
      g_end = g < a.G ? bound_of(a, g + 1) : a.T;
      gc = g < a.G ? a.bcounts + g * a.E : nullptr;
      const float tg = gc ? (float)max(a.blive[g], 1) : 1.0f;
      coef = bc / tg / tg;
#pragma unroll
      for (int j = 0; j < VPL; j++) {
        const int col = col_of<DT, L>(sub, j);
        d[j] = gc && col < a.E ? coef * (float)gc[col] : 0.0f;
      }
    }
    // d at the choices (needed late)
    float dc[KPL];
#pragma unroll
    for (int q = 0; q < KPL; q++) {
      if (q * L >= a.k) break;
      dc[q] = ok && gc && id[q] >= 0 && id[q] < a.E ? coef * (float)gc[id[q]] : 0.0f;
    }
    float m = x[0];
#pragma unroll
    for (int j = 1; j < VPL; j++) m = fmaxf(m, x[j]);
    m = shift_of(lanes_max<L>(m));
    // differences to m first, as all logits may be the type's lowest value (65536 x
    // 256 bf16: 22.5 us, 22.6 with one FMA by Shift, which needs more registers)
    const pair_t c2 = pair(kLog2e, kLog2e), m2 = pair(-m, -m);
    pair_t s2 = pair(0.0f, 0.0f), pd2 = s2;
#pragma unroll
    for (int j = 0; j < VPL; j += 2) {
      const pair_t e = ex2_2(mul2(add2(pair(x[j], x[j + 1]), m2), c2));
      s2 = add2(s2, e);
      pd2 = fma2(e, pair(d[j], d[j + 1]), pd2);
      x[j] = e.x;
      x[j + 1] = e.y;
    }
    const float s = lanes_sum<L>(s2.x + s2.y), inv = rcp(s), lse = m + logf(s);
    float pd = lanes_sum<L>(pd2.x + pd2.y) * inv - zc * lse;
    // the choices: weights and what their gradients give
    float inv_den = inv, dot = 0.0f;
    if (a.dw) {
      float e = 0.0f, ed = 0.0f;
#pragma unroll
      for (int q = 0; q < KPL; q++) {
        if (q * L >= a.k) break;
        xc[q] = ex2((xc[q] - m) * kLog2e);
        e += xc[q];
        ed += xc[q] * dwc[q];
      }
      if (a.renorm) inv_den = rcp(lanes_sum<L>(e));
      dot = lanes_sum<L>(ed) * inv_den;
    }
    if (!a.renorm) pd += dot;
    if (in) {
      T* gp = static_cast<T*>(a.grad) + t * a.gstride;
#pragma unroll
      for (int v = 0; v < VPL / N; v++) {
        float f[N];
        const int col = col_of<DT, L>(sub, v * N);
#pragma unroll
        for (int j = 0; j < N; j++) f[j] = ok ? x[v * N + j] * inv * (d[v * N + j] - pd) : 0.0f;
        if (a.gvec) {
          if (col < a.E) *reinterpret_cast<uint4*>(gp + col) = E::pack(f);
        } else {
#pragma unroll
          for (int j = 0; j < N; j++)
            if (col + j < a.E) gp[col + j] = E::make(f[j]);
        }
      }
    }
    fetch_chosen(t + kStep);
    __syncwarp();
    // their gradients, from fp32, over what was just written
    if (ok && a.dw) {
      T* gp = static_cast<T*>(a.grad) + t * a.gstride;
#pragma unroll
      for (int q = 0; q < KPL; q++) {
        if (q * L >= a.k) break;
        if (id[q] < 0 || id[q] >= a.E) continue;
        gp[id[q]] = E::make(xc[q] * inv * (dc[q] - pd) + xc[q] * inv_den * (a.renorm ? dwc[q] - dot : dwc[q]));
      }
    }
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

bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int check_route(const scape_route_args* q) {
  if (!q) return fail(SCAPE_EINVAL, "args is NULL");
  if (q->dtype < SCAPE_BF16 || q->dtype > SCAPE_F32)
    return fail(SCAPE_EINVAL, "unknown dtype %d", q->dtype);
  if (q->experts < 1 || q->experts > kMaxExperts)
    return fail(SCAPE_EINVAL, "experts=%d outside [1, %d]", q->experts, kMaxExperts);
  if (q->k < 1 || q->k > kMaxK || q->k > q->experts)
    return fail(SCAPE_EINVAL, "k=%d outside [1, min(experts, %d)]", q->k, kMaxK);
  if (q->tokens >= (1ull << 31) || q->row_stride >= (1ull << 32))
    return fail(SCAPE_EINVAL, "tokens must be < 2^31 and row_stride < 2^32");
  if (q->row_stride < (uint64_t)q->experts)
    return fail(SCAPE_EINVAL, "row_stride must be >= experts");
  if (q->n_groups < 1 || q->n_groups >= (1ull << 31) / (uint64_t)q->experts)
    return fail(SCAPE_EINVAL, "n_groups=%llu must be >= 1 and n_groups * experts < 2^31",
                (unsigned long long)q->n_groups);
  return SCAPE_OK;
}

// Lanes of a token for this many experts.
int lanes_of(int experts) {
  int L = 1;
  while (L < 8 && L * 8 < experts) L *= 2;
  return experts <= 256 ? L : experts <= 512 ? 16 : 32;
}

// Tokens of a chunk, in whole rounds of a CTA's warps: at most kChunks of them, two
// CTAs for each of a GB300's 152 SMs.  A constant, as the workspace's size is asked
// for without a device and the order of the sums follows the chunks.
constexpr uint64_t kChunks = 304;

uint64_t chunk_of(const scape_route_args* q) {
  const uint64_t round = (uint64_t)kWarps * 32 / lanes_of(q->experts);
  const uint64_t n = (q->tokens + kChunks - 1) / kChunks;
  return n == 0 ? round : (n + round - 1) / round * round;
}

bool single_chunk(const scape_route_args* q) {
  return q->tokens > 0 && q->tokens <= chunk_of(q) && !q->cu_tokens && q->n_groups == 1;
}

struct Workspace {
  uint64_t slots, nb, part_p, part_c, part_n, part_z, part_b, group_z, done, bytes;
};

Workspace workspace_of(const scape_route_args* q) {
  Workspace w{};
  if (single_chunk(q)) return w;  // one CTA, nothing to hand over
  const uint64_t ch = chunk_of(q);
  w.slots = (q->tokens + ch - 1) / ch + q->n_groups;
  w.nb = (q->experts + kCols - 1) / kCols;
  auto take = [&](uint64_t n) {
    const uint64_t at = w.bytes;
    w.bytes += (n * 4 + 255) / 256 * 256;
    return at;
  };
  w.part_p = take(w.slots * q->experts);
  w.part_c = take(w.slots * q->experts);
  w.part_n = take(w.slots);
  w.part_z = take(w.slots);
  w.part_b = take(q->n_groups * w.nb);
  w.group_z = take(q->n_groups);
  w.done = take(1);
  return w;
}

void fill(const scape_route_args* q, RouteArgs& a) {
  a.x = q->logits;
  a.T = (int64_t)q->tokens;
  a.stride = (int64_t)q->row_stride;
  a.E = q->experts;
  a.k = q->k;
  a.renorm = q->renormalize != 0;
  a.cu = q->cu_tokens;
  a.G = (int64_t)q->n_groups;
  a.valid = q->valid;
  a.chunk = (int64_t)chunk_of(q);
  a.single = single_chunk(q);
  const uint64_t es = q->dtype == SCAPE_F32 ? 4 : 2;
  a.vec = !misaligned(q->logits, 16) && q->row_stride * es % 16 == 0 && q->experts * es % 16 == 0;
}

template <int DT, class LN>
void launch(const RouteArgs& a, unsigned grid, bool back, cudaStream_t s) {
  if (back) {
    route_grad<DT, LN><<<grid, kThreads, 0, s>>>(a);
  } else {  // under 48 KB at every size
    const size_t sm = (size_t)kWarps * LN::ROWS * (LN::CAP + a.k) * 8 + (size_t)(kWarps + 1) * a.E * 4;
    route_chunks<DT, LN><<<grid, kThreads, sm, s>>>(a);
  }
}

template <int DT>
void launch_dt(const RouteArgs& a, unsigned grid, bool back, cudaStream_t s) {
  if (a.E <= 8) launch<DT, Lanes<1, 8, 8>>(a, grid, back, s);
  else if (a.E <= 16) launch<DT, Lanes<2, 8, 8>>(a, grid, back, s);
  else if (a.E <= 32) launch<DT, Lanes<4, 8, 8>>(a, grid, back, s);
  else if (a.E <= 64) launch<DT, Lanes<8, 8, 4>>(a, grid, back, s);
  else if (a.E <= 128) launch<DT, Lanes<8, 16, 4>>(a, grid, back, s);
  else if (a.E <= 256) launch<DT, Lanes<8, 32, 4>>(a, grid, back, s);
  else if (a.E <= 512) launch<DT, Lanes<16, 32, 2>>(a, grid, back, s);
  else launch<DT, Lanes<32, 32, 1>>(a, grid, back, s);
}

void launch_any(int dtype, const RouteArgs& a, unsigned grid, bool back, cudaStream_t s) {
  if (dtype == SCAPE_BF16) launch_dt<SCAPE_BF16>(a, grid, back, s);
  else if (dtype == SCAPE_F16) launch_dt<SCAPE_F16>(a, grid, back, s);
  else launch_dt<SCAPE_F32>(a, grid, back, s);
}

}  // namespace
}  // namespace scape

SCAPE_API int scape_route_workspace(const scape_route_args* args, uint64_t* bytes) {
  using namespace scape;
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  *bytes = 0;
  if (int rc = check_route(args)) return rc;
  *bytes = workspace_of(args).bytes;
  return SCAPE_OK;
}

static int check_route_ptrs(const scape_route_args* q) {
  using namespace scape;
  const uintptr_t es = q->dtype == SCAPE_F32 ? 4 : 2;
  if (q->tokens > 0 && !q->logits) return fail(SCAPE_EINVAL, "logits is NULL");
  if (!q->cu_tokens && q->n_groups != 1) return fail(SCAPE_EINVAL, "n_groups > 1 needs cu_tokens");
  if (misaligned(q->logits, es) || misaligned(q->cu_tokens, 4))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  return SCAPE_OK;
}

SCAPE_API int scape_route(const scape_route_args* args, int32_t* idx, float* weights,
                          int32_t* counts, int32_t* live, float* losses, void* workspace,
                          uint64_t workspace_bytes, void* stream) {
  using namespace scape;
  if (int rc = check_route(args)) return rc;
  if (int rc = check_route_ptrs(args)) return rc;
  if ((args->tokens > 0 && (!idx || !weights)) || !counts || !live || !losses)
    return fail(SCAPE_EINVAL, "idx, weights, counts, live and losses are required");
  if (misaligned(idx, 4) || misaligned(weights, 4) || misaligned(counts, 4) || misaligned(live, 4) ||
      misaligned(losses, 4))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  const Workspace w = workspace_of(args);
  if (w.bytes && (!workspace || misaligned(workspace, 16) || workspace_bytes < w.bytes))
    return fail(SCAPE_EINVAL, "workspace must be %llu bytes, 16-byte aligned",
                (unsigned long long)w.bytes);
  RouteArgs a{};
  fill(args, a);
  char* ws = static_cast<char*>(workspace);
  a.idx = idx;
  a.weights = weights;
  a.counts = counts;
  a.live = live;
  a.losses = losses;
  a.part_p = reinterpret_cast<float*>(ws + w.part_p);
  a.part_c = reinterpret_cast<int32_t*>(ws + w.part_c);
  a.part_n = reinterpret_cast<int32_t*>(ws + w.part_n);
  a.part_z = reinterpret_cast<float*>(ws + w.part_z);
  a.part_b = reinterpret_cast<float*>(ws + w.part_b);
  a.group_z = reinterpret_cast<float*>(ws + w.group_z);
  a.done = reinterpret_cast<uint32_t*>(ws + w.done);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)((args->tokens + a.chunk - 1) / a.chunk);
  launch_any(args->dtype, a, grid ? grid : 1u, false, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SCAPE_ECUDA, "route_chunks: %s", cudaGetErrorString(e));
  if (a.single) return SCAPE_OK;
  // launched behind the chunks: it waits for them on the GPU
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)args->n_groups, (unsigned)w.nb);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, route_finish, a);
  const cudaError_t last = cudaGetLastError();
  if (e == cudaSuccess) e = last;
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "route_finish: %s", cudaGetErrorString(e));
}

SCAPE_API int scape_route_backward(const scape_route_args* args, const int32_t* idx,
                                   const int32_t* counts, const int32_t* live,
                                   const float* d_weights, const float* d_losses, void* grad,
                                   uint64_t grad_stride, void* stream) {
  using namespace scape;
  if (int rc = check_route(args)) return rc;
  if (int rc = check_route_ptrs(args)) return rc;
  if (grad_stride < (uint64_t)args->experts || grad_stride >= (1ull << 32))
    return fail(SCAPE_EINVAL, "grad_stride must be >= experts and < 2^32");
  if (args->tokens == 0) return SCAPE_OK;
  if (!idx || !counts || !live || !grad)
    return fail(SCAPE_EINVAL, "idx, counts, live and grad are required");
  if (grad == args->logits) return fail(SCAPE_EINVAL, "grad must not be the logits");
  const uintptr_t es = args->dtype == SCAPE_F32 ? 4 : 2;
  if (misaligned(idx, 4) || misaligned(counts, 4) || misaligned(live, 4) ||
      misaligned(d_weights, 4) || misaligned(d_losses, 4) || misaligned(grad, es))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  RouteArgs a{};
  fill(args, a);
  a.bidx = idx;
  a.bcounts = counts;
  a.blive = live;
  a.dw = d_weights;
  a.dl = d_losses;
  a.grad = grad;
  a.gstride = (int64_t)grad_stride;
  a.gvec = !misaligned(grad, 16) && grad_stride * es % 16 == 0 && args->experts * es % 16 == 0;
  const unsigned grid = (unsigned)((args->tokens + a.chunk - 1) / a.chunk);
  launch_any(args->dtype, a, grid, true, static_cast<cudaStream_t>(stream));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "route_grad: %s", cudaGetErrorString(e));
}
