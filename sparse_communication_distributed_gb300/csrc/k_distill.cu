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
#include <atomic>
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

constexpr int kMaxCluster = 16;

// Threads of a CTA, CTAs of an SM, vectors of a row that a CTA holds at most,
// for long and for short parts of a row.  Three CTAs share an SM's shared
// memory (twelve of the short kind), and while one waits for its row the others
// compute.
template <int NT_, int MINB_, int PART_>
struct Shape {
  static constexpr int NT = NT_, MINB = MINB_, PART = PART_;
};
using Wide = Shape<512, 3, 4096>;
using Narrow = Shape<128, 12, 1024>;
constexpr int kEnt = 2;  // teacher entries that a thread looks after
static_assert(Wide::NT * kEnt == kMaxK, "every entry has a thread");

// What a row's statistics are made of.  A sum of exponentials is held relative
// to a maximum: s = sum 2^((x - m) c), and s1 the same at temperature 1.
struct Part {
  float m, s, s1;     // coordinates held in registers (with a bucket: those not listed)
  float tm, ts, ts1;  // listed coordinates (bucket only)
  float b;            // over the listed coordinates of this part: sum u_i (t_i - base - s_i), u_i = exp(t_i - base)
  float base, z;      // over all listed coordinates: base = max t_i (u_i then is relative to
                      // teacher_lse with a bucket), z = sum u_i
  float zp;           // sum u_i over those of this part
};
constexpr int kShared = 7;  // the leading members differ from part to part

__device__ __forceinline__ float shfl_max(float x, int n) {
  for (int o = n >> 1; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
__device__ __forceinline__ float shfl_sum(float x, int n) {
  for (int o = n >> 1; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

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

// A cluster of CTAs (often just one) takes a row, each CTA a part of at most
// PART vectors, and reads it once into shared memory; then the cluster takes
// another row.  A thread works only on vectors that it copied itself, so that
// it needs no barrier around them, and in its last pass over a row it starts
// the copy of the next row's vector as soon as it has read the old one.  Each
// thread looks after up to kEnt of the teacher's entries.  TWO: exponentials
// at both temperatures are needed (hard labels at temperature != 1).  BUCKET:
// the coordinates not listed form a bucket; the listed ones are then set to
// -inf in shared memory first and added to the sums by the threads that look
// after them, so that p_rest is a sum and not a difference.
//
// The statistics' buffers are used in turn for one row and the next: between
// two uses of one there are the other row's barriers.
template <int DT, bool TWO, bool BUCKET, class SH>
__global__ __launch_bounds__(SH::NT, SH::MINB) void distill_parts(const DistillArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int EPV = E::kPerVec, NT = SH::NT, kWarps = NT / 32;
  extern __shared__ __align__(16) uint4 buf[];  // the part of the row
  __shared__ Part warps[2][kWarps];
  __shared__ Part parts[2][kMaxCluster];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = a.cluster > 1 ? cluster_rank() : 0;
  const int64_t step = gridDim.x / (unsigned)a.cluster;
  const int64_t v0 = (int64_t)rank * a.part_vecs;
  auto weight_of = [&](int64_t row) { return a.weight ? a.weight[row] : 1.0f; };
  // The part of a row: "here" vectors, whole ones [lo, hi); p is where its first
  // vector starts (outside the row if that is ragged), e0 that coordinate.
  struct Where {
    const T* p;
    int e0, here, lo, hi;
  };
  auto where = [&](int64_t row) {
    const RowView<DT> view(a.x, row * a.stride, a.V);
    const int V = (int)a.V, first = (int)v0 * EPV - view.shift;
    Where w;
    w.e0 = first;
    w.p = view.p + first;
    w.here = max(0, min(a.part_vecs, (V - first + EPV - 1) / EPV));
    w.lo = first < 0 ? 1 : 0;
    w.hi = max(0, min(w.here, (V - first) / EPV));
    return w;
  };
  // starts the copy of one whole vector
  const uint32_t buf_at = (uint32_t)__cvta_generic_to_shared(buf);
  auto fetch = [&](const Where& w, int i) {
    if (i >= w.lo && i < w.hi) copy_async(buf_at + i * 16, w.p + i * EPV);
  };
  // ... and puts ragged ones together from single loads
  auto fetch_ragged = [&](const Where& w) {
    auto one = [&](int i) {
      float f[EPV];
#pragma unroll
      for (int j = 0; j < EPV; j++) {
        const int e = w.e0 + i * EPV + j;
        f[j] = e >= 0 && e < (int)a.V ? E::load(w.p + i * EPV + j) : neg_inf();
      }
      buf[i] = E::pack(f);
    };
    if (w.lo == 1 && w.here > 0 && tid == 0) one(0);
    if (w.here > w.hi && w.here > w.lo && (w.here - 1) % NT == tid) one(w.here - 1);
  };
  if (a.cluster > 1) cluster_arrive();  // "this CTA runs": its shared memory may be written
  bool met = a.cluster == 1;
  int turn = 0;
  int64_t row = blockIdx.x / (unsigned)a.cluster;
  float w = row < a.rows ? weight_of(row) : 0.0f;
  Where at = where(row < a.rows ? row : 0);
  if (w != 0.0f) {
    for (int i = tid; i < at.here; i += NT) fetch(at, i);
    fetch_ragged(at);
  }
  for (; row < a.rows; row += step) {
    const int64_t row2 = row + step;
    const float w_now = w;
    const Where now = at;
    const int here = now.here;
    w = row2 < a.rows ? weight_of(row2) : 0.0f;
    at = where(row2 < a.rows ? row2 : row);
    if (w == 0.0f) at.hi = 0;  // nothing to copy
    T* g = a.grad ? static_cast<T*>(a.grad) + row * a.gstride + now.e0 : nullptr;
    // writes vector i of the part
    const bool same = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(now.p)) & 15u) == 0;
    auto store = [&](int i, const uint4 v) {
      if (same && i >= now.lo && i < now.hi) {
        *reinterpret_cast<uint4*>(g + i * EPV) = v;
      } else {
        const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int j = 0; j < EPV; j++) {
          const int e = now.e0 + i * EPV + j;
          if (e >= 0 && e < (int)a.V) g[i * EPV + j] = t[j];
        }
      }
    };
    if (w_now == 0.0f) {  // the whole cluster agrees
      for (int i = tid; i < here; i += NT)
        if (g) store(i, make_uint4(0, 0, 0, 0));
      for (int i = tid; i < at.hi; i += NT) fetch(at, i);
      if (w != 0.0f) fetch_ragged(at);
      if (a.loss && tid == 0 && rank == 0) a.loss[row] = 0.0f;
      continue;
    }
    // the teacher's entries of this thread: local coordinate (-1: not of this
    // part), t, x
    int el[kEnt];
    float et[kEnt], ex[kEnt];
#pragma unroll
    for (int h = 0; h < kEnt; h++) {
      const int i = h * NT + tid;
      el[h] = -1;
      et[h] = neg_inf();
      ex[h] = 0.0f;
      if (i < a.k) {
        const int32_t e = a.idx[row * a.k + i];
        const float v = load_val(a.vals, a.vals_dtype, row * a.k + i);
        if (e >= a.V) {
          if (a.bad && rank == 0) atomicAdd(a.bad, 1u);
        } else if (e >= 0) {
          et[h] = v / a.tau;
          const int64_t l = (int64_t)e - now.e0;
          if (l >= 0 && l < (int64_t)here * EPV) {
            el[h] = (int)l;
            ex[h] = E::load(now.p + l);
          }
        }
      }
    }
    int64_t y = a.labels ? a.labels[row] : -1;
    if (y >= a.V) {
      if (a.bad && tid == 0 && rank == 0) atomicAdd(a.bad, 1u);
      y = -1;
    }
    const float xy = y >= 0 && tid == 0 ? E::load(now.p + ((int)y - now.e0)) : 0.0f;
    const float tlse = a.tlse ? a.tlse[row] : 0.0f;
    copy_wait();
    if (BUCKET) {
      __syncthreads();
#pragma unroll
      for (int h = 0; h < kEnt; h++)
        if (el[h] >= 0) reinterpret_cast<T*>(buf)[el[h]] = E::make(neg_inf());
      __syncthreads();
    }

    // a thread's statistics, relative to its warp's maximum
    Part q;
    {
      uint4 mx = neg_inf_vec<DT>();
#pragma unroll 4
      for (int i = tid; i < here; i += NT) mx = max_vec<DT>(mx, buf[i]);
      float x[EPV];
      E::unpack(mx, x);
      q.m = x[0];
#pragma unroll
      for (int j = 1; j < EPV; j++) q.m = fmaxf(q.m, x[j]);
      q.m = shfl_max(q.m, 32);
    }
    {
      const float sh = shift_of(q.m);
      const uint64_t c2 = pair(a.c, a.c), mc = pair(-sh * a.c, -sh * a.c);
      const uint64_t l2 = pair(kLog2e, kLog2e), ml = pair(-sh * kLog2e, -sh * kLog2e);
      uint64_t s = 0, s1 = 0;
#pragma unroll 4
      for (int i = tid; i < here; i += NT) {
        float x[EPV];
        E::unpack(buf[i], x);
        if (!g) fetch(at, i);
#pragma unroll
        for (int j = 0; j < EPV; j += 2) {
          const uint64_t xx = pair(x[j], x[j + 1]);
          s = add2(s, ex2_2(fma2(xx, c2, mc)));
          if (TWO) s1 = add2(s1, ex2_2(fma2(xx, l2, ml)));
        }
      }
      const float2 f = unpair(s), f1 = unpair(s1);
      q.s = shfl_sum(f.x + f.y, 32);
      q.s1 = TWO ? shfl_sum(f1.x + f1.y, 32) : q.s;
    }
    q.tm = q.base = neg_inf();
    q.ts = q.ts1 = q.z = q.zp = q.b = 0.0f;
    if (wid * 32 < a.k) {  // the teacher's entries of this warp
      float tmax = et[0], xmax = el[0] >= 0 ? ex[0] : neg_inf();
#pragma unroll
      for (int h = 1; h < kEnt; h++) {
        tmax = fmaxf(tmax, et[h]);
        xmax = fmaxf(xmax, el[h] >= 0 ? ex[h] : neg_inf());
      }
      q.base = shfl_max(tmax, 32);
      const float base = BUCKET ? tlse : shift_of(q.base);
      if (BUCKET) q.tm = shfl_max(xmax, 32);
      const float tsh = shift_of(q.tm);
#pragma unroll
      for (int h = 0; h < kEnt; h++) {
        const float u = expf(et[h] - base);
        q.z += u;
        if (el[h] >= 0) {
          q.zp += u;
          if (u != 0.0f) q.b += u * ((et[h] - base) - ex[h] / a.tau);
          if (BUCKET) {
            q.ts += ex2((ex[h] - tsh) * a.c);
            if (TWO) q.ts1 += ex2((ex[h] - tsh) * kLog2e);
          }
        }
      }
      q.z = shfl_sum(q.z, 32);
      q.b = shfl_sum(q.b, 32);
      if (!BUCKET) q.zp = shfl_sum(q.zp, 32);
      if (BUCKET) {
        q.ts = shfl_sum(q.ts, 32);
        q.ts1 = TWO ? shfl_sum(q.ts1, 32) : q.ts;
      }
    }
    if (lane == 0) warps[turn][wid] = q;
    __syncthreads();
    if (wid == 0) {  // the CTA's
      if (lane < kWarps) q = warps[turn][lane];
      const float base = shfl_max(q.base, kWarps);
      const float m = shfl_max(q.m, kWarps), d = q.m - shift_of(m);
      q.s = shfl_sum(q.s * ex2(d * a.c), kWarps);
      q.s1 = TWO ? shfl_sum(q.s1 * ex2(d * kLog2e), kWarps) : q.s;
      q.m = m;
      if (BUCKET) {
        const float tm = shfl_max(q.tm, kWarps), td = q.tm - shift_of(tm);
        q.ts = shfl_sum(q.ts * ex2(td * a.c), kWarps);
        q.ts1 = TWO ? shfl_sum(q.ts1 * ex2(td * kLog2e), kWarps) : q.ts;
        q.tm = tm;
        q.b = shfl_sum(q.b, kWarps);
        q.z = shfl_sum(q.z, kWarps);
      } else {
        const float bd = shift_of(q.base) - shift_of(base);
        const float f = expf(bd);
        q.b = shfl_sum(q.z == 0.0f ? 0.0f : f * (q.b + bd * q.zp), kWarps);
        q.z = shfl_sum(q.z == 0.0f ? 0.0f : f * q.z, kWarps);
      }
      q.base = base;
      if (lane == 0) {
        parts[turn][rank] = q;
        warps[turn][0] = q;
      }
      if (a.cluster > 1) {
        __syncwarp();
        if (!met) cluster_wait();
        const float* from = reinterpret_cast<const float*>(&warps[turn][0]);
        const float* to = reinterpret_cast<const float*>(&parts[turn][rank]);
        for (int i = lane; i < a.cluster * kShared; i += 32)
          if (i / kShared != (int)rank) put_remote(to + i % kShared, (uint32_t)(i / kShared), from[i % kShared]);
      }
    } else if (!met) {
      cluster_wait();
    }
    met = true;
    if (a.cluster > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    Part t = parts[turn][0];
    for (int i = 1; i < a.cluster; i++) {
      const Part p = parts[turn][i];
      join(t.m, t.s, t.s1, p.m, p.s, p.s1, a.c);
      if (BUCKET) join(t.tm, t.ts, t.ts1, p.tm, p.ts, p.ts1, a.c);
      t.b += p.b;
    }
    t.z = parts[turn][rank].z;
    t.base = parts[turn][rank].base;
    turn ^= 1;
    // the teacher: q_i = exp(t_i - lt), Q = sum q_i
    const bool has = t.base != neg_inf() || t.z != t.z;
    const float lt = BUCKET ? tlse : shift_of(t.base) + logf(t.z);
    const float Q = BUCKET ? t.z : has ? 1.0f : 0.0f;
    // the whole row: all = rest and listed
    float M = t.m, S = t.s, S1 = t.s1;
    if (BUCKET) join(M, S, S1, t.tm, t.ts, t.ts1, a.c);
    const float sh = shift_of(M), shr = shift_of(t.m);
    const bool bucket = BUCKET && has && t.s > 0.0f;
    const float qr = bucket ? fmaxf(0.0f, 1.0f - Q) : 0.0f;
    if (a.loss && tid == 0 && rank == 0) {
      const float L = sh / a.tau + logf(S);
      float l = 0.0f;
      if (has) {  // sum q_i (t_i - lt - s_i) + L sum q_i
        float kl = BUCKET ? t.b + Q * L : t.b / t.z + (L - logf(t.z));
        if (qr > 0.0f) {  // log q_rest - log p_rest, both from what is listed
          const float odds = t.ts / t.s * ex2((shift_of(t.tm) - shr) * a.c);
          const float logp = odds < 1.0f ? log1pf(odds) : L - (shr / a.tau + logf(t.s));
          kl += qr * (log1pf(-Q) + logp);
        }
        l = a.kd * a.tau * a.tau * kl;
      }
      if (y >= 0) l += a.ce * (sh + logf(S1) - xy);
      a.loss[row] = w_now * l;
    }
    if (!g) {
      if (w != 0.0f) fetch_ragged(at);
      continue;
    }
    // gradient = K1 2^((x - m) c) + K2 2^((x - m) log2 e), m the maximum of
    // what the buffer holds; the listed coordinates and the label after that
    const float A = has ? w_now * a.kd * a.tau : 0.0f, C1 = y >= 0 ? w_now * a.ce : 0.0f;
    float K1 = A * Q / S, K2 = C1 / S1;
    if (BUCKET) {
      const float pr = t.s * ex2((shr - sh) * a.c) / S;
      const float pr1 = t.s1 * ex2((shr - sh) * kLog2e) / S1;
      const float ptop = t.ts * ex2((shift_of(t.tm) - sh) * a.c) / S;
      const float d = qr > 0.0f ? Q - ptop : Q * pr;  // (Q + q_rest) p_rest - q_rest; Q + q_rest = 1
      K1 = t.s > 0.0f ? A * d / t.s : 0.0f;
      K2 = t.s1 > 0.0f ? C1 * pr1 / t.s1 : 0.0f;
    }
    if (!TWO) K1 += K2;
    const uint64_t c2 = pair(a.c, a.c), mc = pair(-shr * a.c, -shr * a.c), k1 = pair(K1, K1);
    const uint64_t l2 = pair(kLog2e, kLog2e), ml = pair(-shr * kLog2e, -shr * kLog2e);
    const uint64_t k2 = pair(K2, K2);
    auto grad_of = [&](uint64_t x) {
      uint64_t v = mul2(k1, ex2_2(fma2(x, c2, mc)));
      if (TWO) v = fma2(k2, ex2_2(fma2(x, l2, ml)), v);
      return v;
    };
#pragma unroll 2
    for (int i = tid; i < here; i += NT) {
      float x[EPV];
      E::unpack(buf[i], x);
      fetch(at, i);
#pragma unroll
      for (int j = 0; j < EPV; j += 2) {
        const float2 f = unpair(grad_of(pair(x[j], x[j + 1])));
        x[j] = f.x;
        x[j + 1] = f.y;
      }
      store(i, E::pack(x));
    }
    if (w != 0.0f) fetch_ragged(at);
    const int64_t ly = y - now.e0;
    const bool y_here = y >= 0 && ly >= 0 && ly < (int64_t)here * EPV;
    bool y_listed = false;
#pragma unroll
    for (int h = 0; h < kEnt; h++) y_listed |= y_here && el[h] == ly;
    y_listed = __syncthreads_or(y_listed);
#pragma unroll
    for (int h = 0; h < kEnt; h++) {
      if (el[h] < 0) continue;
      const float d = ex[h] - sh, u = has ? expf(et[h] - lt) : 0.0f;
      float v = A * ((Q + qr) * ex2(d * a.c) / S - u);
      if (y >= 0) v += C1 * ex2(d * kLog2e) / S1;
      if (y_here && el[h] == ly) v -= C1;
      g[el[h]] = E::make(v);
    }
    if (y_here && !y_listed && tid == 0) g[ly] = E::make(unpair(grad_of(pair(xy, xy))).x - C1);
  }
  if (!met) cluster_wait();
}

template <int DT, bool TWO, bool BUCKET, class SH>
cudaError_t launch_parts(const DistillArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};  // the shared-memory opt-in is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(distill_parts<DT, TWO, BUCKET, SH>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, SH::PART * 16);
    if (e == cudaSuccess)  // clusters of 16
      e = cudaFuncSetAttribute(distill_parts<DT, TWO, BUCKET, SH>,
                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  // as many clusters as the GPU holds at once, evened out over the rounds
  const int64_t slots = (int64_t)num_sms() * SH::MINB / a.cluster;
  const int64_t rounds = (a.rows + slots - 1) / slots;
  const int64_t clusters = (a.rows + rounds - 1) / rounds;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * a.cluster));
  cfg.blockDim = dim3(SH::NT);
  cfg.dynamicSmemBytes = (size_t)a.part_vecs * 16;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)a.cluster;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, distill_parts<DT, TWO, BUCKET, SH>, a);
}

template <int DT, class SH>
cudaError_t launch_sized(const DistillArgs& a, cudaStream_t s) {
  const bool two = a.labels && a.tau != 1.0f, bucket = a.tlse != nullptr;
  if (two) return bucket ? launch_parts<DT, true, true, SH>(a, s) : launch_parts<DT, true, false, SH>(a, s);
  return bucket ? launch_parts<DT, false, true, SH>(a, s) : launch_parts<DT, false, false, SH>(a, s);
}

template <int DT>
cudaError_t launch_distill(DistillArgs& a, cudaStream_t s) {
  // vectors of a row at most: one more where rows start inside one
  constexpr int64_t EPV = Elem<DT>::kPerVec;
  const bool whole = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.stride % EPV == 0;
  const int64_t nv = (a.V + (whole ? 0 : EPV - 1) + EPV - 1) / EPV;
  cudaError_t e;
  if (nv > (int64_t)Wide::PART * kMaxCluster) {
    const int64_t cap = (int64_t)num_sms() * 4;
    distill_rows<DT><<<(unsigned)(a.rows < cap ? a.rows : cap), kThreads, 0, s>>>(a);
    e = cudaSuccess;
  } else {
    a.cluster = 1;
    while (nv > (int64_t)Wide::PART * a.cluster) a.cluster *= 2;
    // few rows: more CTAs for each, down to a vector or two a thread
    while (a.cluster < 8 && a.rows * a.cluster * 2 <= num_sms() && nv > Narrow::NT * 2 * a.cluster)
      a.cluster *= 2;
    a.part_vecs = (int)((nv + a.cluster - 1) / a.cluster);
    const bool narrow = a.part_vecs <= Narrow::PART && a.k <= Narrow::NT * kEnt;
    e = narrow ? launch_sized<DT, Narrow>(a, s) : launch_sized<DT, Wide>(a, s);
  }
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
