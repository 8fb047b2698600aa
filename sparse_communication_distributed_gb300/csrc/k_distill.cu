// Distillation from a teacher's top logits with an optional hard label: the
// loss of every row and the gradient of the student's logits.
//
// With s = x / tau, p = softmax(s), L = log sum exp(s), the teacher's q_i at
// the listed coordinates and q_rest for all others together,
//   KL = sum_i q_i (log q_i - (s_i - L)) + q_rest (log q_rest - (L_rest - L))
//   d KL / d s_j = p_j (sum q + q_rest) - q_j                      j listed
//                = p_j (sum q + q_rest) - q_rest exp(s_j - L_rest) j not listed
// where L_rest = log sum exp(s) over the coordinates not listed.  L_rest is
// summed over just those, not taken as a difference, so that a student which is
// sure of the listed words keeps its exact small p_rest.  Every coordinate is
// written by the formula of the unlisted ones and the k listed ones (and the
// label) are then set one by one from fp32 values, so each gradient is rounded
// once.
//
// A CTA takes a row: one pass for the running maxima and sums, one for the
// gradient.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "objective.cuh"
#include "scape_kernels.cuh"

#define SCAPE_API extern "C" __attribute__((visibility("default")))

namespace scape {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxK = 1024;
constexpr int kFilter = 32768;  // bits: coordinates that may be listed, modulo this

struct DistillArgs {
  const void* x;
  void* grad;
  const int32_t* idx;
  const void* vals;
  const float* tlse;
  const int64_t* labels;
  const float* weight;
  float* loss;
  uint32_t* bad;
  int64_t rows, V, stride, gstride;
  int k, vals_dtype;
  float tau, c;  // temperature, log2(e) / temperature
  float kd, ce;
  int cluster, part_vecs;  // CTAs of a row, vectors of each one's part
};

__device__ __forceinline__ float load_val(const void* p, int dtype, int64_t i) {
  if (dtype == SCAPE_F32) return static_cast<const float*>(p)[i];
  const uint16_t* h = static_cast<const uint16_t*>(p) + i;
  return dtype == SCAPE_BF16 ? Elem<SCAPE_BF16>::load(h) : Elem<SCAPE_F16>::load(h);
}

// Running maximum and sum of exponentials of c * x.
struct Lse {
  float m = neg_inf(), s = 0.0f;
  __device__ __forceinline__ void add(float x, float c) {
    if (x > m) {
      s *= ex2((shift_of(m) - x) * c);
      m = x;
    }
    s += ex2((x - shift_of(m)) * c);
  }
};

template <int DT>
__global__ __launch_bounds__(kThreads) void distill_rows(const DistillArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int EPV = E::kPerVec;
  __shared__ int32_t sidx[kMaxK];  // -1: empty
  __shared__ float sq[kMaxK], sx[kMaxK];
  __shared__ uint32_t filter[kFilter / 32];
  __shared__ float fbuf[32];
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const RowView<DT> view(a.x, row * a.stride, a.V);
    const int64_t nv = view.vectors();
    T* g = a.grad ? static_cast<T*>(a.grad) + row * a.gstride : nullptr;
    const float w = a.weight ? a.weight[row] : 1.0f;
    if (w == 0.0f) {
      if (g)
        for (int64_t e = tid; e < a.V; e += kThreads) g[e] = E::make(0.0f);
      if (a.loss && tid == 0) a.loss[row] = 0.0f;
      continue;
    }
    // the teacher's entries
    for (int i = tid; i < kFilter / 32; i += kThreads) filter[i] = 0;
    __syncthreads();
    float tm = neg_inf();
    for (int i = tid; i < a.k; i += kThreads) {
      int32_t e = a.idx[row * a.k + i];
      float t = neg_inf();
      if (e >= a.V) {
        if (a.bad) atomicAdd(a.bad, 1u);
        e = -1;
      }
      if (e >= 0) {
        t = load_val(a.vals, a.vals_dtype, row * a.k + i) / a.tau;
        sx[i] = E::load(view.p + e);
        atomicOr(&filter[e % kFilter / 32], 1u << (e & 31));
      } else {
        e = -1;
        sx[i] = 0.0f;
      }
      sidx[i] = e;
      sq[i] = t;
      if (!(t <= tm)) tm = t;  // NaN stays
    }
    int64_t y = a.labels ? a.labels[row] : -1;
    if (y >= a.V) {
      if (a.bad && tid == 0) atomicAdd(a.bad, 1u);
      y = -1;
    }
    const float xy = y >= 0 ? E::load(view.p + y) : 0.0f;
    const bool tail_mode = a.tlse != nullptr;
    bool has = __syncthreads_or(tm != neg_inf());
    float lt = 0.0f;  // log of the teacher's normaliser
    if (has) {
      if (tail_mode) {
        lt = a.tlse[row];
      } else {
        const float M = shift_of(cta_max(tm, fbuf));
        float z = 0.0f;
        for (int i = tid; i < a.k; i += kThreads) z += expf(sq[i] - M);
        lt = M + logf(cta_sum(z, fbuf));
      }
    }
    float qs = 0.0f;
    for (int i = tid; i < a.k; i += kThreads) {
      const float logq = sq[i] - lt, q = has && sidx[i] >= 0 ? expf(logq) : 0.0f;
      sq[i] = q;
      qs += q;
    }
    const float Q = cta_sum(qs, fbuf);

    // statistics of the row
    Lse all, rest, one;  // over s: every coordinate, those not listed; over x
    for (int64_t v = tid; v < nv; v += kThreads) {
      float x[EPV];
      E::unpack(view.load(v), x);
      const int64_t e0 = view.first_of(v);
#pragma unroll
      for (int j = 0; j < EPV; j++) {
        const int64_t e = e0 + j;
        if (e < 0 || e >= a.V) continue;
        all.add(x[j], a.c);
        if (y >= 0) one.add(x[j], kLog2e);
        if (tail_mode) {
          bool listed = (filter[e % kFilter / 32] >> (e & 31)) & 1u;
          if (listed) {
            listed = false;
            for (int i = 0; i < a.k; i++) listed |= sidx[i] == e;
          }
          if (!listed) rest.add(x[j], a.c);
        }
      }
    }
    const float Ms = shift_of(cta_max(all.m, fbuf));
    const float L = Ms / a.tau + logf(cta_sum(all.s * ex2((shift_of(all.m) - Ms) * a.c), fbuf));
    float L1 = 0.0f, Lr = neg_inf();
    if (y >= 0)
      L1 = Ms + logf(cta_sum(one.s * ex2((shift_of(one.m) - Ms) * kLog2e), fbuf));
    if (tail_mode) {
      const float Mr = shift_of(cta_max(rest.m, fbuf));
      Lr = Mr / a.tau + logf(cta_sum(rest.s * ex2((shift_of(rest.m) - Mr) * a.c), fbuf));
    }
    const bool bucket = tail_mode && has && Lr > neg_inf();
    const float qr = bucket ? fmaxf(0.0f, 1.0f - Q) : 0.0f;
    float kl = 0.0f;
    for (int i = tid; i < a.k; i += kThreads) {
      const float q = sq[i];
      if (q != 0.0f)
        kl += q * ((load_val(a.vals, a.vals_dtype, row * a.k + i) / a.tau - lt) - (sx[i] / a.tau - L));
    }
    kl = cta_sum(kl, fbuf);
    if (qr > 0.0f) kl += qr * (logf(qr) - (Lr - L));
    if (a.loss && tid == 0) {
      float l = has ? a.kd * a.tau * a.tau * kl : 0.0f;
      if (y >= 0) l += a.ce * (L1 - xy);
      a.loss[row] = w * l;
    }
    if (!g) continue;

    // the gradient: ref = L or L_rest, so that exp(s - ref) keeps the small
    // probabilities of a bucket
    const float A = has ? w * a.kd * a.tau : 0.0f, C1 = y >= 0 ? w * a.ce : 0.0f;
    const float ref = bucket ? Lr : L;
    const float C = bucket ? A * ((Q + qr) * expf(Lr - L) - qr) : A * Q;
    const float ref2 = ref * kLog2e, L12 = L1 * kLog2e;
    auto grad_of = [&](float x) {
      float r = C * ex2(x * a.c - ref2);
      if (y >= 0) r += C1 * ex2(x * kLog2e - L12);
      return r;
    };
    __syncthreads();  // sx is complete: the row may be overwritten
    for (int64_t v = tid; v < nv; v += kThreads) {
      float x[EPV];
      E::unpack(view.load(v), x);
      const int64_t e0 = view.first_of(v);
#pragma unroll
      for (int j = 0; j < EPV; j++)
        if (e0 + j >= 0 && e0 + j < a.V) g[e0 + j] = E::make(grad_of(x[j]));
    }
    __syncthreads();
    bool label_listed = false;
    for (int i = tid; i < a.k; i += kThreads) {
      if (sidx[i] < 0) continue;
      float r = A * ((Q + qr) * expf(sx[i] / a.tau - L) - sq[i]);
      if (y >= 0) {
        r += C1 * expf(sx[i] - L1);
        if (sidx[i] == y) {
          r -= C1;
          label_listed = true;
        }
      }
      g[sidx[i]] = E::make(r);
    }
    label_listed = __syncthreads_or(label_listed);
    if (y >= 0 && !label_listed && tid == 0) g[y] = E::make(grad_of(xy) - C1);
    __syncthreads();
  }
}

// ---- Rows held on chip -------------------------------------------------------

constexpr int kVecs = 8;                     // vectors of a row that a thread holds
constexpr int kPart = kThreads * kVecs;      // vectors of a row that a CTA holds
constexpr int kMaxCluster = 8;
constexpr int kWarps = kThreads / 32;

// What a row's statistics are made of.  A sum of exponentials is held relative
// to a maximum: sum 2^((x - m) c), and sum1 the same at temperature 1.
struct Part {
  float m, s, s1;        // coordinates held in registers (with a bucket: those not listed)
  float tm, ts, ts1;     // listed coordinates (bucket only)
  float a;               // sum q_i (log q_i - s_i) over the listed coordinates of this part
};

__device__ __forceinline__ void join(float& m, float& s, float& s1, float m2, float s2, float s12,
                                     float c) {
  const float M = fmaxf(m, m2), sh = shift_of(M);
  const float f = ex2((m - sh) * c), f2 = ex2((m2 - sh) * c);
  const float g = ex2((m - sh) * kLog2e), g2 = ex2((m2 - sh) * kLog2e);
  s = s * f + s2 * f2;
  s1 = s1 * g + s12 * g2;
  m = M;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Writes to the same place of another CTA's shared memory in the cluster.
__device__ __forceinline__ void put_remote(const float* local, uint32_t rank, float v) {
  uint32_t at = (uint32_t)__cvta_generic_to_shared(local), there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
}

// A cluster of CTAs takes a row, each a part of at most kPart vectors, and
// reads it once.  TWO: the exponentials at both temperatures are needed (hard
// labels at temperature != 1).  BUCKET: the coordinates not listed form a
// bucket; the listed ones are then taken out of the registers first and added
// to the sums from the list, so that p_rest is a sum and not a difference.
template <int DT, bool TWO, bool BUCKET>
__global__ __launch_bounds__(kThreads, 2) void distill_parts(const DistillArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int EPV = E::kPerVec;
  __shared__ int32_t sidx[kMaxK];  // local coordinate in this part, -1: not here
  __shared__ float sq[kMaxK], sx[kMaxK];
  __shared__ uint32_t listed[BUCKET ? kPart * 8 / 32 : 1];  // a byte for each vector
  __shared__ Part warps[kWarps];
  __shared__ Part parts[kMaxCluster];
  __shared__ float steacher[2];  // sum of q; whether there is any
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = a.cluster > 1 ? cluster_rank() : 0;
  const int64_t row = blockIdx.x / (unsigned)a.cluster;
  const RowView<DT> view(a.x, row * a.stride, a.V);
  const int64_t nv = view.vectors();
  const int64_t v0 = (int64_t)rank * a.part_vecs;
  const int here = (int)max((int64_t)0, min((int64_t)a.part_vecs, nv - v0));  // vectors of this part
  const int64_t e0 = view.first_of(v0);  // coordinate of the part's first element (may be < 0)
  T* g = a.grad ? static_cast<T*>(a.grad) + row * a.gstride : nullptr;
  const float w = a.weight ? a.weight[row] : 1.0f;
  const bool same = g && ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(view.p)) & 15u) == 0;

  auto store = [&](int i, const float (&f)[EPV]) {  // local vector i
    const int64_t e = e0 + (int64_t)i * EPV;
    if (same && e >= 0 && e + EPV <= a.V) {
      *reinterpret_cast<uint4*>(g + e) = E::pack(f);
    } else {
#pragma unroll
      for (int j = 0; j < EPV; j++)
        if (e + j >= 0 && e + j < a.V) g[e + j] = E::make(f[j]);
    }
  };
  if (w == 0.0f) {  // the whole cluster agrees
    const float zero[EPV] = {};
    if (g)
      for (int i = tid; i < here; i += kThreads) store(i, zero);
    if (a.loss && tid == 0 && rank == 0) a.loss[row] = 0.0f;
    return;
  }
  if (a.cluster > 1) cluster_arrive();  // "this CTA runs": its shared memory may be written

  uint4 r[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; u++) {
    const int i = u * kThreads + tid;
    r[u] = i < here ? view.load(v0 + i) : make_uint4(E::kNegInf2, E::kNegInf2, E::kNegInf2, E::kNegInf2);
  }
  int64_t y = a.labels ? a.labels[row] : -1;
  if (y >= a.V) {
    if (a.bad && tid == 0 && rank == 0) atomicAdd(a.bad, 1u);
    y = -1;
  }
  if (BUCKET) {
    for (int i = tid; i < kPart * 8 / 32; i += kThreads) listed[i] = 0;
    __syncthreads();
    for (int i = tid; i < a.k; i += kThreads) {
      const int32_t e = a.idx[row * a.k + i];
      const int64_t l = e - e0;
      if (e >= 0 && e < a.V && l >= 0 && l < (int64_t)here * EPV) {
        const int bit = (int)(l / EPV) * 8 + (int)(l % EPV);
        atomicOr(&listed[bit >> 5], 1u << (bit & 31));
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kVecs; u++) {
      const uint32_t bits = reinterpret_cast<const uint8_t*>(listed)[u * kThreads + tid];
      if (bits) {
        float x[EPV];
        E::unpack(r[u], x);
#pragma unroll
        for (int j = 0; j < EPV; j++)
          if (bits >> j & 1) x[j] = neg_inf();
        r[u] = E::pack(x);
      }
    }
  }

  // the teacher: one warp, all entries; x at those of this part
  Part mine{neg_inf(), 0.0f, 0.0f, neg_inf(), 0.0f, 0.0f, 0.0f};
  if (wid == 0) {
    float tm = neg_inf();
    for (int i = lane; i < a.k; i += 32) {
      const int32_t e = a.idx[row * a.k + i];
      const int64_t l = e - e0;
      float t = neg_inf();
      bool in = false;
      if (e >= a.V) {
        if (a.bad && rank == 0) atomicAdd(a.bad, 1u);
      } else if (e >= 0) {
        t = load_val(a.vals, a.vals_dtype, row * a.k + i) / a.tau;
        in = l >= 0 && l < (int64_t)here * EPV;
        if (in) sx[i] = E::load(view.p + e);
      }
      sidx[i] = in ? (int32_t)l : -1;
      sq[i] = t;
      if (!(t <= tm)) tm = t;  // NaN stays
    }
    const bool has = __any_sync(kFull, tm != neg_inf());
    float lt = 0.0f;
    if (has) {
      if (a.tlse) {
        lt = a.tlse[row];
      } else {
#pragma unroll
        for (int o = 16; o; o >>= 1) tm = fmaxf(tm, __shfl_xor_sync(kFull, tm, o));
        tm = shift_of(tm);
        float z = 0.0f;
        for (int i = lane; i < a.k; i += 32) z += expf(sq[i] - tm);
#pragma unroll
        for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
        lt = tm + logf(z);
      }
    }
    float Q = 0.0f;
    for (int i = lane; i < a.k; i += 32) {
      const float logq = sq[i] - lt, q = has ? expf(logq) : 0.0f;
      sq[i] = q;
      Q += q;
      if (sidx[i] < 0) continue;
      const float x = sx[i];
      if (q != 0.0f) mine.a += q * (logq - x / a.tau);
      if (BUCKET) join(mine.tm, mine.ts, mine.ts1, x, 1.0f, 1.0f, a.c);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      Q += __shfl_xor_sync(kFull, Q, o);
      mine.a += __shfl_xor_sync(kFull, mine.a, o);
      if (BUCKET) {
        const float m2 = __shfl_xor_sync(kFull, mine.tm, o), s2 = __shfl_xor_sync(kFull, mine.ts, o),
                    s12 = __shfl_xor_sync(kFull, mine.ts1, o);
        join(mine.tm, mine.ts, mine.ts1, m2, s2, s12, a.c);
      }
    }
    if (lane == 0) {
      steacher[0] = Q;
      steacher[1] = has ? 1.0f : 0.0f;
    }
  }
  const float xy = y >= 0 && tid == 0 ? E::load(view.p + y) : 0.0f;

  // the part's statistics: a thread's, its warp's, the CTA's, the cluster's
  {
    float m = neg_inf();
#pragma unroll
    for (int u = 0; u < kVecs; u++) {
      float x[EPV];
      E::unpack(r[u], x);
#pragma unroll
      for (int j = 0; j < EPV; j++) m = fmaxf(m, x[j]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    const float sh = shift_of(m), mc = sh * a.c, mc1 = sh * kLog2e;
    float s = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int u = 0; u < kVecs; u++) {
      float x[EPV];
      E::unpack(r[u], x);
#pragma unroll
      for (int j = 0; j < EPV; j++) {
        s += ex2(fmaf(x[j], a.c, -mc));
        if (TWO) s1 += ex2(fmaf(x[j], kLog2e, -mc1));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      s += __shfl_xor_sync(kFull, s, o);
      if (TWO) s1 += __shfl_xor_sync(kFull, s1, o);
    }
    mine.m = m;
    mine.s = s;
    mine.s1 = TWO ? s1 : s;
  }
  if (lane == 0) warps[wid] = mine;
  __syncthreads();
  if (wid == 0) {
    Part q = warps[lane < kWarps ? lane : 0];
    if (lane >= kWarps) q = Part{neg_inf(), 0.0f, 0.0f, neg_inf(), 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float m2 = __shfl_xor_sync(kFull, q.m, o), s2 = __shfl_xor_sync(kFull, q.s, o),
                  s12 = __shfl_xor_sync(kFull, q.s1, o);
      join(q.m, q.s, q.s1, m2, s2, s12, a.c);
    }
    if (lane == 0) {
      q.tm = warps[0].tm;
      q.ts = warps[0].ts;
      q.ts1 = warps[0].ts1;
      q.a = warps[0].a;
      warps[0] = q;
      if (a.cluster == 1) parts[0] = q;
    }
    if (a.cluster > 1) {
      __syncwarp();
      cluster_wait();
      const float* from = reinterpret_cast<const float*>(&warps[0]);
      const float* to = reinterpret_cast<const float*>(&parts[rank]);
      for (int i = lane; i < a.cluster * 7; i += 32) put_remote(to + i % 7, (uint32_t)(i / 7), from[i % 7]);
    }
  } else if (a.cluster > 1) {
    cluster_wait();
  }
  if (a.cluster > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  Part t = parts[0];
  for (int i = 1; i < a.cluster; i++) {
    const Part q = parts[i];
    join(t.m, t.s, t.s1, q.m, q.s, q.s1, a.c);
    if (BUCKET) join(t.tm, t.ts, t.ts1, q.tm, q.ts, q.ts1, a.c);
    t.a += q.a;
  }
  // the whole row: all = rest and listed
  const float Q = steacher[0];
  const bool has = steacher[1] != 0.0f;
  float M = t.m, S = t.s, S1 = t.s1;
  if (BUCKET) join(M, S, S1, t.tm, t.ts, t.ts1, a.c);
  const float sh = shift_of(M), shr = shift_of(t.m);
  const bool bucket = BUCKET && has && t.s > 0.0f;
  const float qr = bucket ? fmaxf(0.0f, 1.0f - Q) : 0.0f;
  if (a.loss && tid == 0 && rank == 0) {
    const float L = sh / a.tau + logf(S);
    float l = 0.0f;
    if (has) {
      float kl = t.a + Q * L;
      if (qr > 0.0f) {  // log q_rest - log p_rest, both from what is listed
        const float odds = t.ts / t.s * ex2((shift_of(t.tm) - shr) * a.c);
        const float logp = odds < 1.0f ? log1pf(odds) : L - (shr / a.tau + logf(t.s));
        kl += qr * (log1pf(-Q) + logp);
      }
      l = a.kd * a.tau * a.tau * kl;
    }
    if (y >= 0) l += a.ce * (sh + logf(S1) - xy);
    a.loss[row] = w * l;
  }
  if (!g) return;

  // gradient = K1 2^((x - m) c) + K2 2^((x - m) log2 e), m the maximum of what
  // the registers hold; the listed coordinates and the label after that
  const float A = has ? w * a.kd * a.tau : 0.0f, C1 = y >= 0 ? w * a.ce : 0.0f;
  float K1 = A * Q / S, K2 = C1 / S1;
  if (BUCKET) {
    const float pr = t.s * ex2((shr - sh) * a.c) / S, pr1 = t.s1 * ex2((shr - sh) * kLog2e) / S1;
    const float ptop = t.ts * ex2((shift_of(t.tm) - sh) * a.c) / S;
    const float d = qr > 0.0f ? Q - ptop : Q * pr;  // (Q + q_rest) p_rest - q_rest, as Q + q_rest = 1
    K1 = t.s > 0.0f ? A * d / t.s : 0.0f;
    K2 = t.s1 > 0.0f ? C1 * pr1 / t.s1 : 0.0f;
  }
  if (!TWO) K1 += K2;
  const float mc = shr * a.c, mc1 = shr * kLog2e;
  auto grad_of = [&](float x) {
    float v = K1 * ex2(fmaf(x, a.c, -mc));
    if (TWO) v = fmaf(K2, ex2(fmaf(x, kLog2e, -mc1)), v);
    return v;
  };
#pragma unroll
  for (int u = 0; u < kVecs; u++) {
    const int i = u * kThreads + tid;
    if (i < here) {
      float x[EPV];
      E::unpack(r[u], x);
#pragma unroll
      for (int j = 0; j < EPV; j++) x[j] = grad_of(x[j]);
      store(i, x);
    }
  }
  const int64_t ly = y - e0;
  const bool y_here = y >= 0 && ly >= 0 && ly < (int64_t)here * EPV;
  bool y_listed = false;
  float x_y = 0.0f;
  if (y_here && tid == 0) x_y = xy;
  __syncthreads();
  for (int i = tid; i < a.k; i += kThreads) {
    if (sidx[i] < 0) continue;
    const float d = sx[i] - sh;
    float v = A * ((Q + qr) * ex2(d * a.c) / S - sq[i]);
    if (y >= 0) v += C1 * ex2(d * kLog2e) / S1;
    if (y_here && sidx[i] == ly) {
      v -= C1;
      y_listed = true;
    }
    g[e0 + sidx[i]] = E::make(v);
  }
  if (y_here) {  // the same for the whole CTA
    y_listed = __syncthreads_or(y_listed);
    if (!y_listed && tid == 0) g[y] = E::make(grad_of(x_y) - C1);
  }
}

template <int DT, bool TWO, bool BUCKET>
cudaError_t launch_parts(const DistillArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.rows * a.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)a.cluster;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, distill_parts<DT, TWO, BUCKET>, a);
}

template <int DT>
cudaError_t launch_distill(DistillArgs& a, cudaStream_t s) {
  // vectors of a row, one more where it starts inside one
  const int64_t nv = a.V / Elem<DT>::kPerVec + 2;
  if (nv > (int64_t)kPart * kMaxCluster) {
    const int64_t cap = (int64_t)num_sms() * 4;
    distill_rows<DT><<<(unsigned)(a.rows < cap ? a.rows : cap), kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  a.cluster = 1;
  while (nv > (int64_t)kPart * a.cluster) a.cluster *= 2;
  a.part_vecs = (int)((nv + a.cluster - 1) / a.cluster);
  const bool two = a.labels && a.tau != 1.0f, bucket = a.tlse != nullptr;
  cudaError_t e;
  if (two) e = bucket ? launch_parts<DT, true, true>(a, s) : launch_parts<DT, true, false>(a, s);
  else e = bucket ? launch_parts<DT, false, true>(a, s) : launch_parts<DT, false, false>(a, s);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
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

bool known(int dtype) { return dtype >= SCAPE_BF16 && dtype <= SCAPE_F32; }
bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

}  // namespace
}  // namespace scape

SCAPE_API int scape_distill_loss(const scape_distill_args* args, void* stream) {
  using namespace scape;
  if (!args) return fail(SCAPE_EINVAL, "args is NULL");
  const scape_distill_args& q = *args;
  if (!known(q.dtype)) return fail(SCAPE_EINVAL, "unknown dtype %d", q.dtype);
  if (q.vocab < 1 || q.vocab >= (1ull << 31))
    return fail(SCAPE_EINVAL, "vocab=%llu must be in [1, 2^31)", (unsigned long long)q.vocab);
  if (q.k < 0 || q.k > kMaxK) return fail(SCAPE_EINVAL, "k=%d outside [0, %d]", q.k, kMaxK);
  if (q.k > 0 && !known(q.vals_dtype))
    return fail(SCAPE_EINVAL, "unknown vals_dtype %d", q.vals_dtype);
  if (q.rows >= (1ull << 31) || q.row_stride >= (1ull << 32) || q.grad_stride >= (1ull << 32))
    return fail(SCAPE_EINVAL, "rows must be < 2^31 and strides < 2^32");
  if (q.row_stride < q.vocab) return fail(SCAPE_EINVAL, "row_stride must be >= vocab");
  if (q.grad && q.grad_stride < q.vocab) return fail(SCAPE_EINVAL, "grad_stride must be >= vocab");
  if (!(q.temperature > 0.0f) || !std::isfinite(q.temperature) ||
      !std::isfinite(kLog2e / q.temperature))
    return fail(SCAPE_EINVAL, "temperature must be finite and > 0");
  if (!std::isfinite(q.kd_weight) || !std::isfinite(q.ce_weight))
    return fail(SCAPE_EINVAL, "kd_weight and ce_weight must be finite");
  if (!q.loss && !q.grad) return fail(SCAPE_EINVAL, "loss or grad is required");
  if (q.rows == 0) return SCAPE_OK;
  if (!q.logits) return fail(SCAPE_EINVAL, "logits is NULL");
  if (q.k > 0 && (!q.idx || !q.vals)) return fail(SCAPE_EINVAL, "idx and vals are required");
  const uintptr_t es = q.dtype == SCAPE_F32 ? 4 : 2, vs = q.vals_dtype == SCAPE_F32 ? 4 : 2;
  if (misaligned(q.logits, es) || misaligned(q.grad, es) || misaligned(q.idx, 4) ||
      misaligned(q.vals, vs) || misaligned(q.teacher_lse, 4) || misaligned(q.labels, 8) ||
      misaligned(q.row_weight, 4) || misaligned(q.loss, 4) || misaligned(q.bad_count, 4))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  if (q.grad == q.logits && q.grad_stride != q.row_stride)
    return fail(SCAPE_EINVAL, "an in-place gradient needs grad_stride == row_stride");
  DistillArgs a{};
  a.x = q.logits;
  a.grad = q.grad;
  a.idx = q.idx;
  a.vals = q.vals;
  a.tlse = q.k > 0 ? q.teacher_lse : nullptr;
  a.labels = q.labels;
  a.weight = q.row_weight;
  a.loss = q.loss;
  a.bad = q.bad_count;
  a.rows = (int64_t)q.rows;
  a.V = (int64_t)q.vocab;
  a.stride = (int64_t)q.row_stride;
  a.gstride = (int64_t)q.grad_stride;
  a.k = q.k;
  a.vals_dtype = q.vals_dtype;
  a.tau = q.k > 0 ? q.temperature : 1.0f;  // without a teacher only the cross entropy is left
  a.c = kLog2e / a.tau;
  a.kd = q.kd_weight;
  a.ce = q.ce_weight;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = q.dtype == SCAPE_BF16  ? launch_distill<SCAPE_BF16>(a, s)
                        : q.dtype == SCAPE_F16 ? launch_distill<SCAPE_F16>(a, s)
                                               : launch_distill<SCAPE_F32>(a, s);
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "distill: %s", cudaGetErrorString(e));
}
