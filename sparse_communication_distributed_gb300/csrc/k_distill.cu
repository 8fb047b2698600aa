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
// sure of the listed words keeps its exact small p_rest, in the loss and in the
// gradient (rest_of).  Every coordinate is
// written by the formula of the unlisted ones and the k listed ones (and the
// label) are then set one by one from fp32 values, so each gradient is rounded
// once.
//
// Rows of up to 884736 16-bit words or 442368 fp32 ones are held on chip, each by
// a CTA or a cluster of them, and move through HBM once (distill_parts); longer
// ones are read twice, once for the running maxima and sums and once for the
// gradient (distill_rows).
//
// The bound is HBM where a row is short enough for three CTAs an SM: 8192 x 32000
// bf16 with the gradient take 187 us, 5.6 TB/s, 83 % of the copy bandwidth (DRAM
// busy 64 % and issue active 59 % on 4096 rows, which fit the caches in part).
// Rows of 50257 take two CTAs of 105 KB: 313 us for 8192 with bucket and labels
// (78 %), 84 us for the loss alone of 4096 (72 %).  There neither limit is reached
// (issue 58 %, DRAM 56 %, 29 % of the warps; the instructions alone are 45 us): 20
// warps an SM do not cover the chain of copy, maximum, sums and merge.  Rows of
// 131072 fp32 words take eight CTAs, whose exchange costs a cluster barrier a row:
// 156 us for 768 (76 %).  Rows of a vector or two a thread are bound by that chain
// too (16384 x 1003 bf16 80 us, barriers first among the stalls); Narrow's 64
// registers spill 168 to 192 bytes a thread, outside the loops over vectors.
// Rows that do not fit the chip are read twice and written an element at a time:
// 64 x 1000003 bf16 take 1.03 ms, 4 % of the copy bandwidth.
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

constexpr int kThreads = 512;
constexpr int kMaxK = 1024;
constexpr int kFilter = 32768;  // bits: coordinates that may be listed, modulo this

// What all coordinates not listed get together, in units of kd tau:
// (Q + q_rest) p_rest - q_rest, which is Q - p_listed as well where Q + q_rest = 1.
// Of the two differences the one of the smaller numbers keeps more of a small
// result: a student and a teacher both sure of the listed words have p_rest and
// q_rest near 0, both unsure Q and p_listed.
__device__ __forceinline__ float rest_of(float Q, float q_rest, float p_listed, float p_rest) {
  return q_rest > 0.0f && p_rest > 0.5f ? Q - p_listed : (Q + q_rest) * p_rest - q_rest;
}

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
      s *= ex2((m - x) * c);
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
      float v = neg_inf();
      if (e >= a.V) {
        if (a.bad) atomicAdd(a.bad, 1u);
        e = -1;
      }
      if (e >= 0) {
        v = load_val(a.vals, a.vals_dtype, row * a.k + i);
        sx[i] = E::load(view.p + e);
        atomicOr(&filter[e % kFilter / 32], 1u << (e & 31));
      } else {
        e = -1;
        sx[i] = 0.0f;
      }
      sidx[i] = e;
      sq[i] = v;
      if (!(v <= tm)) tm = v;  // NaN stays
    }
    int64_t y = a.labels ? a.labels[row] : -1;
    if (y >= a.V) {
      if (a.bad && tid == 0) atomicAdd(a.bad, 1u);
      y = -1;
    }
    const float xy = y >= 0 ? E::load(view.p + y) : 0.0f;
    const bool tail_mode = a.tlse != nullptr;
    bool has = __syncthreads_or(tm != neg_inf());
    // log q = (v - base) / tau - lz (v / tau alone may be beyond fp32)
    float base = 0.0f, lz = 0.0f;
    if (has) {
      if (tail_mode) {
        lz = a.tlse[row];
      } else {
        base = shift_of(cta_max(tm, fbuf));
        float z = 0.0f;
        for (int i = tid; i < a.k; i += kThreads) z += expf((sq[i] - base) / a.tau);
        lz = logf(cta_sum(z, fbuf));
      }
    }
    float qs = 0.0f;
    for (int i = tid; i < a.k; i += kThreads) {
      const float logq = (sq[i] - base) / a.tau - lz, q = has && sidx[i] >= 0 ? expf(logq) : 0.0f;
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
    const float S = cta_sum(all.s * ex2((all.m - Ms) * a.c), fbuf), ls = logf(S);
    float S1 = 1.0f, Mr = 0.0f, Sr = 0.0f;
    if (y >= 0) S1 = cta_sum(one.s * ex2((one.m - Ms) * kLog2e), fbuf);
    if (tail_mode) {
      Mr = shift_of(cta_max(rest.m, fbuf));
      Sr = cta_sum(rest.s * ex2((rest.m - Mr) * a.c), fbuf);
    }
    const bool bucket = tail_mode && has && Sr > 0.0f;
    const float qr = bucket ? fmaxf(0.0f, 1.0f - Q) : 0.0f;
    float kl = 0.0f, top = 0.0f;
    for (int i = tid; i < a.k; i += kThreads) {
      const float q = sq[i];
      if (bucket && sidx[i] >= 0) top += ex2((sx[i] - Ms) * a.c);
      if (q != 0.0f)
        kl += q * (((load_val(a.vals, a.vals_dtype, row * a.k + i) - base) / a.tau - lz) - ((sx[i] - Ms) / a.tau - ls));
    }
    kl = cta_sum(kl, fbuf);
    if (bucket) top = cta_sum(top, fbuf) / S;
    if (qr > 0.0f) kl += qr * (logf(qr) - ((Mr - Ms) / a.tau + logf(Sr) - ls));
    if (a.loss && tid == 0) {
      float l = has ? a.kd * a.tau * a.tau * kl : 0.0f;
      if (y >= 0) l += a.ce * (Ms - xy + logf(S1));
      a.loss[row] = w * l;
    }
    if (!g) continue;

    // the gradient: p = exp(s - ref) / over with the maximum and the sum of the row, or
    // of the bucket, whose small probabilities it keeps; from differences to the
    // maximum, as a maximum may be the type's lowest value and p still 1 / vocab
    const float A = has ? w * a.kd * a.tau : 0.0f, C1 = y >= 0 ? w * a.ce : 0.0f;
    const float ref = bucket ? Mr : Ms, over = bucket ? Sr : S;
    const float C = has ? A * (bucket ? rest_of(Q, qr, top, Sr * ex2((Mr - Ms) * a.c) / S) : Q) / over : 0.0f;
    const float C2 = C1 / S1;
    auto grad_of = [&](float x) {
      float r = C * ex2((x - ref) * a.c);
      if (y >= 0) r += C2 * ex2((x - Ms) * kLog2e);
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
      float r = has ? A * ((Q + qr) * (ex2((sx[i] - Ms) * a.c) / S) - sq[i]) : 0.0f;
      if (y >= 0) {
        r += C2 * ex2((sx[i] - Ms) * kLog2e);
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

constexpr int kMaxCluster = 8;

// Threads of a CTA, vectors of a row that each of them has at most, CTAs of an
// SM, teacher entries that a thread looks after.  Three CTAs with parts of up to
// 64 KB share an SM's shared memory, and while one waits for its row the others
// compute; two with parts of 105 KB do better where that saves a cluster, eight
// with parts of 16 KB share an SM where rows are short or few, and there is one shape for many entries.
template <int NT_, int VECS_, int MINB_, int ENT_, bool DIFF_ = false>
struct Shape {
  static constexpr int NT = NT_, MINB = MINB_, ENT = ENT_;
  static constexpr bool DIFF = DIFF_;  // Terms (gradient of 16384 x 1003 bf16 with labels and bucket: 82 us
                                       // with differences, 87 without; of 8192 x 50257 319 and 312)
  static constexpr int PART = NT_ * VECS_, MAXK = NT_ * ENT_;
  static constexpr int MOST = 13824;  // vectors that fit at all (216 KB)
};
using Wide = Shape<256, 16, 3, 1>;
using Large = Shape<320, 21, 2, 1>;
using Narrow = Shape<128, 8, 8, 2, true>;
using Deep = Shape<320, 21, 2, 4>;
static_assert(Deep::MAXK >= kMaxK, "every entry has a thread");

// What a row's statistics are made of.  A sum of exponentials is held relative
// to a maximum: s = sum 2^((x - m) c), and s1 the same at temperature 1.
struct Part {
  float m, s, s1;     // coordinates held in registers (with a bucket: those not listed)
  float tm, ts, ts1;  // listed coordinates (the sums with a bucket only)
  float b;            // over the listed coordinates of this part: sum u_i (log u_i - (x_i - tm) / tau): no
                      // term holds a maximum, which may be the type's lowest value
  float zp;           // sum u_i over those
  float base, z;      // over all listed coordinates: base = max vals_i and z = sum u_i, where log u_i =
                      // (vals_i - base) / tau, or vals_i / tau - teacher_lse with a bucket
};
constexpr int kShared = 8;  // the leading members differ from part to part

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

enum { kOne, kTwo, kSquare };

// What one warp works out for all threads once a row's statistics are known.
struct __align__(16) Row {
  float m, K1, K2, rS;         // gradient = K1 2^((x - m) c) + K2 2^((x - m) log2 e) at unlisted, by Terms
  float M, A, C1, rS1;         // p = 2^((x - M) c) rS; softmax(x) = 2^((x - M) log2 e) rS1
  float Qr, base, rz, unused;  // sum q + q_rest; q_i = exp(log_u(vals_i, base)) rz
};

// What a row's loss is worked out from.
struct Loss {
  float M, m, S, S1;   // as in Part and Row: the whole row's sums
  float z, Q, qr;      // the teacher's
  float top, s, b;     // p_listed on the scale of s; as in Part, relative to M
  float w, xy;
  int64_t row;
  bool has, hard;
};

// A cluster of CTAs (often just one) takes a row, each CTA a part of at most
// PART vectors, and reads it once into shared memory; then the cluster takes
// another row.  A thread works only on vectors that it copied itself, so that
// it needs no barrier around them, and in its last pass over a row it starts
// the copy of the next row's vector as soon as it has read the old one.  Each
// thread looks after up to ENT of the teacher's entries.  EXPS: whether
// exponentials at temperature 1 are needed as well (hard labels at another
// temperature), and whether they are squares of the others (temperature 2: a
// fifth of the instructions less; of 8192 x 50257 with labels and bucket 348 -> 317 us, its loss alone, 4096
// rows, 98 -> 87 us).
// BUCKET: the coordinates not listed form a bucket; the listed ones are then set
// to -inf in shared memory first and added to the sums by the threads that look
// after them, so that p_rest is a sum and not a difference.
//
// The statistics' buffers are used in turn for one row and the next: between
// two uses of one there are the other row's barriers.
template <int DT, int EXPS, bool BUCKET, class SH>
__global__ __launch_bounds__(SH::NT, SH::MINB) void distill_parts(const DistillArgs a) {
  constexpr bool TWO = EXPS != kOne;
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int EPV = E::kPerVec, NT = SH::NT, ENT = SH::ENT;
  constexpr int kWarps = NT / 32, kMerge = kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : 16;
  static_assert(kWarps <= 16, "a warp merges the others' statistics");
  constexpr int BLK = 2;  // vectors that a thread handles at a time
  extern __shared__ __align__(16) uint4 buf[];  // the part of the row
  __shared__ Part warps[2][kWarps];
  __shared__ Part parts[2][kMaxCluster];
  __shared__ Row rows[2];
  __shared__ Loss pend[32];  // rows whose losses are still to be worked out, a lane each
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = a.cluster > 1 ? cluster_rank() : 0;
  const int64_t step = gridDim.x / (unsigned)a.cluster;
  const int v0 = (int)rank * a.part_vecs;
  const int V = (int)a.V;
  const float inv_tau = 1.0f / a.tau;
  auto weight_of = [&](int64_t row) { return a.weight ? a.weight[row] : 1.0f; };
  // The part of a row: "here" vectors, whole ones [lo, hi); p is where its first
  // vector starts (outside the row if that is ragged), e0 that coordinate.
  struct Where {
    const T* p;
    int e0, here, lo, hi;
  };
  auto where = [&](const T* row_start) {
    Where w;
    w.e0 = v0 * EPV - (int)((reinterpret_cast<uintptr_t>(row_start) & 15u) / sizeof(T));
    w.p = row_start + w.e0;
    const int left = V - w.e0;  // elements from the part's start
    w.here = max(0, min(a.part_vecs, (left + EPV - 1) / EPV));
    w.lo = w.e0 < 0 ? 1 : 0;
    w.hi = max(0, min(w.here, left / EPV));
    return w;
  };
  const uint32_t buf_at = (uint32_t)__cvta_generic_to_shared(buf) + tid * 16;
  // starts the copies of the whole vectors among BLK of this thread's (w.hi is 0
  // for a row that is not read)
  auto fetch = [&](const Where& w, int u0) {
    const T* p = w.p + (int64_t)(u0 * NT + tid) * EPV;
    const uint32_t to = buf_at + u0 * NT * 16;
    if (u0 * NT >= w.lo && (u0 + BLK) * NT <= w.hi) {
#pragma unroll
      for (int u = 0; u < BLK; u++) copy_async(to + u * NT * 16, p + u * NT * EPV);
    } else {
#pragma unroll
      for (int u = 0; u < BLK; u++) {
        const int i = (u0 + u) * NT + tid;
        if (i >= w.lo && i < w.hi) copy_async(to + u * NT * 16, p + u * NT * EPV);
      }
    }
  };
  // ... and puts ragged ones together from single loads
  auto fetch_ragged = [&](const Where& w) {
    auto one = [&](int i) {
      float f[EPV];
#pragma unroll
      for (int j = 0; j < EPV; j++) {
        const int e = w.e0 + i * EPV + j;
        f[j] = e >= 0 && e < V ? E::load(w.p + i * EPV + j) : neg_inf();
      }
      buf[i] = E::pack(f);
    };
    if (w.lo == 1 && w.here > 0 && tid == 0) one(0);
    if (w.here > w.hi && w.here > w.lo && (w.here - 1) % NT == tid) one(w.here - 1);
  };
  // Side inputs of a row: what the arrays hold, loaded a row ahead, and what
  // that and x make of it once the row is in shared memory.
  int32_t raw_e[ENT];
  float raw_v[ENT], raw_lse = 0.0f;
  int64_t raw_y = -1;
  auto load_side = [&](int64_t row) {
#pragma unroll
    for (int h = 0; h < ENT; h++) {
      const int i = h * NT + tid;
      raw_e[h] = -1;
      raw_v[h] = 0.0f;
      if (i < a.k) {
        raw_e[h] = a.idx[row * a.k + i];
        raw_v[h] = load_val(a.vals, a.vals_dtype, row * a.k + i);
      }
    }
    if (a.labels) raw_y = a.labels[row];
    if (BUCKET) raw_lse = a.tlse[row];
  };
  // the teacher's entries of this thread: local coordinate (-1: not of this
  // part), vals, x; the label and, for one thread, x there
  int el[ENT], y = -1;
  float et[ENT], ex[ENT], xy = 0.0f, tlse = 0.0f;
  auto take_side = [&](const Where& w) {
#pragma unroll
    for (int h = 0; h < ENT; h++) {
      const int32_t e = raw_e[h];
      el[h] = -1;
      et[h] = neg_inf();
      ex[h] = 0.0f;
      if (e >= V) {
        if (a.bad && rank == 0) atomicAdd(a.bad, 1u);
      } else if (e >= 0) {
        et[h] = raw_v[h];
        const int l = e - w.e0;  // e < 2^20, e0 > -8
        if (l >= 0 && l < w.here * EPV) {
          el[h] = l;
          // (from shared memory where a barrier comes before the copies of the
          // next row that follow)
          ex[h] = E::load((BUCKET || a.grad ? reinterpret_cast<const T*>(buf) : w.p) + l);
        }
      }
    }
    if (raw_y >= V && a.bad && tid == 0 && rank == 0) atomicAdd(a.bad, 1u);
    y = raw_y < 0 || raw_y >= V ? -1 : (int)raw_y;
    if (y >= 0 && tid == 0) xy = E::load(w.p + (y - w.e0));
    tlse = raw_lse;
  };
  auto log_u = [&](float v, float base) { return BUCKET ? v * inv_tau - base : (v - base) * inv_tau; };
  auto row_at = [&](int64_t row) { return static_cast<const T*>(a.x) + row * a.stride; };
  // writes vector i of a part of a gradient's row that starts at g
  auto put = [&](T* g, const Where& w, bool same, int i, const uint4 v) {
    T* p = g + i * EPV;
    if (same && i >= w.lo && i < w.hi) {
      *reinterpret_cast<uint4*>(p) = v;
    } else if (i < w.here) {
      const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int j = 0; j < EPV; j++) {
        const int e = w.e0 + i * EPV + j;
        if (e >= 0 && e < V) p[j] = t[j];
      }
    }
  };
  auto grad_at = [&](int64_t row, const Where& w) {
    return a.grad ? static_cast<T*>(a.grad) + row * a.gstride + w.e0 : nullptr;
  };
  auto alike = [](const T* g, const T* p) {  // in vectors at the same places
    return ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(p)) & 15u) == 0;
  };
  // a row of weight 0
  auto fill = [&](int64_t row) {
    const Where w = where(row_at(row));
    T* const g = grad_at(row, w);
    const bool same = alike(g, w.p);
    if (g)
      for (int i = tid; i < w.here; i += NT) put(g, w, same, i, make_uint4(0, 0, 0, 0));
    if (a.loss && tid == 0 && rank == 0) a.loss[row] = 0.0f;
  };
  // The losses of up to 32 rows at once, by the first warp: their logarithms and
  // quotients would hold up the CTA if one lane worked them out for each row.
  int n_pend = 0;
  auto write_losses = [&]() {
    __syncwarp();
    if (lane < n_pend) {
      const Loss p = pend[lane];
      const float ls = logf(p.S);
      float l = 0.0f;
      if (p.has) {  // sum q_i (log u_i - log z - (x_i - M) / tau) + log S sum q_i
        float kl = BUCKET ? p.b + p.Q * ls : p.b / p.z + (ls - logf(p.z));
        if (p.qr > 0.0f) {  // log q_rest - log p_rest, both from what is listed
          const float odds = p.top / p.s;
          const float logp = odds < 1.0f ? log1pf(odds) : (p.M - p.m) * inv_tau + (ls - logf(p.s));
          kl += p.qr * (log1pf(-p.Q) + logp);
        }
        l = a.kd * a.tau * a.tau * kl;
      }
      if (p.hard) l += a.ce * (p.M - p.xy + logf(p.S1));
      a.loss[p.row] = p.w * l;
    }
    __syncwarp();
    n_pend = 0;
  };
  auto weight_or_1 = [&](int64_t row) { return row < a.rows ? weight_of(row) : 1.0f; };
  if (a.cluster > 1) cluster_arrive_relaxed();  // "this CTA runs": its shared memory may be written
  bool met = a.cluster == 1;
  int turn = 0;
  // (the whole cluster agrees on which rows are read)
  int64_t row = blockIdx.x / (unsigned)a.cluster;
  float w = weight_or_1(row);
  while (w == 0.0f) {
    fill(row);
    row += step;
    w = weight_or_1(row);
  }
  bool more = row < a.rows;  // a row to copy: this one, then the next that is read
  Where at = where(row_at(more ? row : 0));
  // starts the copies of that row that the blocks of a pass did not reach
  auto fetch_rest = [&](int u0) {
    for (; u0 * NT < at.hi; u0 += BLK) fetch(at, u0);
    if (more) fetch_ragged(at);
  };
  if (more) {
    load_side(row);
    fetch_rest(0);
  }
  while (row < a.rows) {
    const float w_now = w;
    const Where now = at;
    const int here = now.here;
    int64_t row2 = row + step;
    w = weight_or_1(row2);
    T* const g = grad_at(row, now);
    const bool same = alike(g, now.p);
    copy_wait();
    __syncthreads();
    take_side(now);
    if (BUCKET) {  // (each listed place is read and written by one thread)
#pragma unroll
      for (int h = 0; h < ENT; h++)
        if (el[h] >= 0) reinterpret_cast<T*>(buf)[el[h]] = E::make(neg_inf());
      __syncthreads();
    }
    // Calls f(vector, u) for all vectors of this thread: in whole blocks of BLK,
    // with ahead(u0) between a block's loads and its work, then one by one, -inf
    // beyond the part, by the warps that have any.  Returns the u after the blocks.
    auto each = [&](auto ahead, auto f) {
      int u0 = 0;
#pragma unroll 1
      for (; (u0 + BLK) * NT <= here; u0 += BLK) {
        uint4 r[BLK];
#pragma unroll
        for (int u = 0; u < BLK; u++) r[u] = buf[(u0 + u) * NT + tid];
        ahead(u0);
#pragma unroll
        for (int u = 0; u < BLK; u++) f(r[u], u0 + u);
      }
#pragma unroll 1
      for (int u = u0; u * NT + wid * 32 < here; u++) {
        const int i = u * NT + tid;
        f(i < here ? buf[i] : neg_inf_vec<DT>(), u);
      }
      return u0;
    };

    // a thread's statistics, relative to its warp's maximum
    Part q;
    {
      uint4 mx = neg_inf_vec<DT>();
      each([](int) {}, [&](const uint4 r, int) { mx = max_vec<DT>(mx, r); });
      float x[EPV];
      E::unpack(mx, x);
      q.m = x[0];
#pragma unroll
      for (int j = 1; j < EPV; j++) q.m = fmaxf(q.m, x[j]);
      q.m = shfl_max(q.m, 32);
    }
    // the next row that is read
    while (w == 0.0f) {
      row2 += step;
      w = weight_or_1(row2);
    }
    more = row2 < a.rows;
    at = where(row_at(more ? row2 : row));
    if (more) load_side(row2);
    else at.hi = 0;
    {
      // (this warp's own maximum, far below the row's where all it has is masked)
      const float sh = shift_of(q.m);
      const Terms<SH::DIFF> at_tau(sh, a.c), at_1(sh, kLog2e);
      pair_t s = pair(0.0f, 0.0f), s1 = s;
      const int u0 = each([&](int u0) { if (!g) fetch(at, u0); },
                          [&](const uint4 r, int) {
        float x[EPV];
        E::unpack(r, x);
#pragma unroll
        for (int j = 0; j < EPV; j += 2) {
          const pair_t xx = pair(x[j], x[j + 1]), e = at_tau(xx);
          s = add2(s, e);
          if (EXPS == kTwo) s1 = add2(s1, at_1(xx));
          if (EXPS == kSquare) s1 = fma2(e, e, s1);
        }
      });
      if (!g) fetch_rest(u0);
      q.s = shfl_sum(s.x + s.y, 32) * at_tau.undo;
      q.s1 = TWO ? shfl_sum(s1.x + s1.y, 32) * (EXPS == kTwo ? at_1.undo : at_tau.undo * at_tau.undo) : q.s;
    }
    q.tm = q.base = neg_inf();
    q.ts = q.ts1 = q.z = q.zp = q.b = 0.0f;
    if (wid * 32 < a.k) {  // the teacher's entries of this warp
      float tmax = et[0], xmax = el[0] >= 0 ? ex[0] : neg_inf();
#pragma unroll
      for (int h = 1; h < ENT; h++) {
        tmax = fmaxf(tmax, et[h]);
        xmax = fmaxf(xmax, el[h] >= 0 ? ex[h] : neg_inf());
      }
      q.base = shfl_max(tmax, 32);
      const float base = BUCKET ? tlse : shift_of(q.base);
      q.tm = shfl_max(xmax, 32);
      const float tsh = shift_of(q.tm);
#pragma unroll
      for (int h = 0; h < ENT; h++) {
        const float lu = log_u(et[h], base), u = expf(lu);
        q.z += u;
        if (el[h] >= 0) {
          q.zp += u;
          if (u != 0.0f) q.b += u * (lu - (ex[h] - tsh) * inv_tau);
          if (BUCKET) {
            q.ts += ex2((ex[h] - tsh) * a.c);
            if (TWO) q.ts1 += ex2((ex[h] - tsh) * kLog2e);
          }
        }
      }
      q.z = shfl_sum(q.z, 32);
      q.b = shfl_sum(q.b, 32);
      q.zp = shfl_sum(q.zp, 32);
      if (BUCKET) {
        q.ts = shfl_sum(q.ts, 32);
        q.ts1 = TWO ? shfl_sum(q.ts1, 32) : q.ts;
      }
    }
    if (lane == 0) warps[turn][wid] = q;
    __syncthreads();
    if (wid == 0) {
      // b relative to another logit instead of tm
      auto raise = [&](float to) {
        if (q.zp != 0.0f) q.b += q.zp * ((shift_of(to) - shift_of(q.tm)) * inv_tau);
      };
      // the CTA's, then the cluster's: the partial statistics of n parts, one in
      // each of the first n lanes
      auto merge = [&](int n) {
        const float m = shfl_max(q.m, n), d = q.m - shift_of(m);
        q.s = shfl_sum(q.s * ex2(d * a.c), n);
        q.s1 = TWO ? shfl_sum(q.s1 * ex2(d * kLog2e), n) : q.s;
        q.m = m;
        const float tm = shfl_max(q.tm, n), td = q.tm - shift_of(tm);
        if (BUCKET) {
          q.ts = shfl_sum(q.ts * ex2(td * a.c), n);
          q.ts1 = TWO ? shfl_sum(q.ts1 * ex2(td * kLog2e), n) : q.ts;
        }
        raise(tm);
        q.tm = tm;
        q.b = shfl_sum(q.b, n);
        q.zp = shfl_sum(q.zp, n);
      };
      q = warps[turn][min(lane, kWarps - 1)];
      if (lane >= kWarps) q = Part{neg_inf(), 0.0f, 0.0f, neg_inf(), 0.0f, 0.0f, 0.0f, 0.0f, neg_inf(), 0.0f};
      const float base = shfl_max(q.base, kMerge);
      if (!BUCKET) {  // relative to the CTA's base
        const float bd = (shift_of(q.base) - shift_of(base)) * inv_tau, f = expf(bd);
        // (f = 0: a warp of entries at the type's lowest value, whose q are 0 whatever its b)
        q.b = f == 0.0f || q.z == 0.0f ? 0.0f : f * (q.b + bd * q.zp);
        q.z = q.z == 0.0f ? 0.0f : f * q.z;
        q.zp = q.zp == 0.0f ? 0.0f : f * q.zp;
      }
      merge(kMerge);
      const float z = shfl_sum(q.z, kMerge);
      if (a.cluster > 1) {
        if (lane == 0) {
          warps[turn][0] = q;
          parts[turn][rank] = q;
        }
        __syncwarp();
        if (!met) cluster_wait();
        const float* from = reinterpret_cast<const float*>(&warps[turn][0]);
        const float* to = reinterpret_cast<const float*>(&parts[turn][rank]);
        for (int i = lane; i < a.cluster * kShared; i += 32)
          if (i / kShared != (int)rank) put_remote(to + i % kShared, (uint32_t)(i / kShared), from[i % kShared]);
        cluster_arrive();
        cluster_wait();
        q = parts[turn][min(lane, a.cluster - 1)];
        if (lane >= a.cluster) {
          q.m = q.tm = neg_inf();
          q.s = q.s1 = q.ts = q.ts1 = q.b = q.zp = 0.0f;
        }
        merge(kMaxCluster);
      }
      if (lane == 0) {
        // the teacher: q_i = u_i / z (u_i with a bucket), Q = sum q_i
        const bool has = base != neg_inf() || z != z;
        const float Q = BUCKET ? z : has ? 1.0f : 0.0f;
        // the whole row: all = rest and listed
        float M = q.m, S = q.s, S1 = q.s1;
        if (BUCKET) join(M, S, S1, q.tm, q.ts, q.ts1, a.c);
        const float sh = shift_of(M), shr = shift_of(q.m);
        const bool bucket = BUCKET && has && q.s > 0.0f;
        const float qr = bucket ? fmaxf(0.0f, 1.0f - Q) : 0.0f;
        if (g) {
          Row r;
          r.M = sh;
          r.m = shr;
          r.rS = has ? rcp(S) : 0.0f;  // (infinite where the mask leaves no word: not for a term that is not there)
          r.rS1 = y >= 0 ? rcp(S1) : 0.0f;
          r.A = has ? w_now * a.kd * a.tau : 0.0f;
          r.C1 = y >= 0 ? w_now * a.ce : 0.0f;
          r.Qr = Q + qr;
          r.base = BUCKET ? tlse : shift_of(base);
          r.rz = !has ? 0.0f : BUCKET ? 1.0f : rcp(z);
          r.unused = 0.0f;
          r.K1 = r.A * Q * r.rS;
          r.K2 = r.C1 * r.rS1;
          if (BUCKET) {
            const float f = ex2((shr - sh) * a.c), f1 = ex2((shr - sh) * kLog2e);
            const float top = q.ts * ex2((q.tm - sh) * a.c) * r.rS;
            r.K1 = q.s > 0.0f ? r.A * rest_of(Q, qr, top, q.s * f * r.rS) / q.s : 0.0f;
            r.K2 = q.s1 > 0.0f ? r.C1 * f1 * r.rS1 : 0.0f;
          }
          if (!TWO) r.K1 += r.K2;
          const float undo = Terms<SH::DIFF>(shr, a.c).undo;
          r.K1 *= undo;
          if (TWO) r.K2 *= EXPS == kTwo ? Terms<SH::DIFF>(shr, kLog2e).undo : undo * undo;
          rows[turn] = r;
        }
        if (a.loss && rank == 0) {
          raise(M);
          pend[n_pend] = {sh, shr, S, S1, z, Q, qr, BUCKET ? q.ts * ex2((q.tm - shr) * a.c) : 0.0f,
                          q.s, q.b, w_now, xy, row, has, y >= 0};
        }
      }
      if (a.loss && rank == 0 && ++n_pend == 32) write_losses();
    } else if (a.cluster > 1) {
      if (!met) cluster_wait();
      cluster_arrive_relaxed();
      cluster_wait();
    }
    met = true;
    if (g) {
      __syncthreads();
      const Row t = rows[turn];
      const Terms<SH::DIFF> at_tau(t.m, a.c), at_1(t.m, kLog2e);
      const pair_t k1 = pair(t.K1, t.K1), k2 = pair(t.K2, t.K2);
      auto grad_of = [&](pair_t x) {
        const pair_t e = at_tau(x);
        if (EXPS == kSquare) return mul2(e, fma2(k2, e, k1));
        const pair_t v = mul2(k1, e);
        return EXPS == kTwo ? fma2(k2, at_1(x), v) : v;
      };
      const int u0 = each([&](int u0) { fetch(at, u0); },
                          [&](const uint4 r, int u) {
        float x[EPV];
        E::unpack(r, x);
#pragma unroll
        for (int j = 0; j < EPV; j += 2) {
          const pair_t f = grad_of(pair(x[j], x[j + 1]));
          x[j] = f.x;
          x[j + 1] = f.y;
        }
        put(g, now, same, u * NT + tid, E::pack(x));
      });
      fetch_rest(u0);
      const int ly = y - now.e0;
      const bool y_here = y >= 0 && ly >= 0 && ly < here * EPV;
      bool y_listed = false;
#pragma unroll
      for (int h = 0; h < ENT; h++) y_listed |= y_here && el[h] == ly;
      y_listed = __syncthreads_or(y_listed);
#pragma unroll
      for (int h = 0; h < ENT; h++) {
        if (el[h] < 0) continue;
        const float d = ex[h] - t.M;
        float v = t.A * (t.Qr * ex2(d * a.c) * t.rS - expf(log_u(et[h], t.base)) * t.rz);
        v += t.C1 * ex2(d * kLog2e) * t.rS1;
        if (y_here && el[h] == ly) v -= t.C1;
        g[el[h]] = E::make(v);
      }
      if (y_here && !y_listed && tid == 0) g[ly] = E::make(grad_of(pair(xy, xy)).x - t.C1);
    }
    for (row += step; row < min(row2, a.rows); row += step) fill(row);
    row = row2;
    turn ^= 1;
  }
  if (wid == 0 && n_pend) write_losses();
  if (!met) cluster_wait();
}

template <int DT, int EXPS, bool BUCKET, class SH>
cudaError_t launch_parts(const DistillArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};  // the shared-memory opt-in is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(distill_parts<DT, EXPS, BUCKET, SH>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, SH::MOST * 16);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(num_sms() * a.cluster));
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
  // as many clusters as the GPU holds at once, evened out over the rounds.  A
  // cluster lies within a GPC, so that is less than the CTAs it holds divided by
  // the cluster's (51 of 8, not 57), and one too many would run after all others.
  int slots = 0;
  if (a.cluster > 1) {
    e = cudaOccupancyMaxActiveClusters(&slots, distill_parts<DT, EXPS, BUCKET, SH>, &cfg);
    if (e != cudaSuccess) return e;
  } else {
    slots = num_sms() * std::min(SH::MINB, 224 * 1024 / (a.part_vecs * 16 + 4096));
  }
  slots = std::max(slots, 1);
  const int64_t rounds = (a.rows + slots - 1) / slots;
  cfg.gridDim.x = (unsigned)((a.rows + rounds - 1) / rounds * a.cluster);
  return cudaLaunchKernelEx(&cfg, distill_parts<DT, EXPS, BUCKET, SH>, a);
}

template <int DT, class SH>
cudaError_t launch_sized(const DistillArgs& a, cudaStream_t s) {
  const bool bucket = a.tlse != nullptr;
  if (!a.labels || a.tau == 1.0f)
    return bucket ? launch_parts<DT, kOne, true, SH>(a, s) : launch_parts<DT, kOne, false, SH>(a, s);
  if (a.tau == 2.0f)
    return bucket ? launch_parts<DT, kSquare, true, SH>(a, s) : launch_parts<DT, kSquare, false, SH>(a, s);
  return bucket ? launch_parts<DT, kTwo, true, SH>(a, s) : launch_parts<DT, kTwo, false, SH>(a, s);
}

template <int DT>
cudaError_t launch_distill(DistillArgs& a, cudaStream_t s) {
  // vectors of a row at most: one more where rows start inside one
  constexpr int64_t EPV = Elem<DT>::kPerVec;
  const bool whole = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.stride % EPV == 0;
  const int64_t nv = (a.V + (whole ? 0 : EPV - 1) + EPV - 1) / EPV;
  cudaError_t e;
  if (nv > (int64_t)Wide::MOST * kMaxCluster) {
    const int64_t cap = (int64_t)num_sms() * 4;
    distill_rows<DT><<<(unsigned)(a.rows < cap ? a.rows : cap), kThreads, 0, s>>>(a);
    e = cudaSuccess;
  } else {
    // large parts where one or two hold the row (gradient of 1000 x 50257 bf16: 54
    // us against 59 with two wide ones, x 100000: 98 against 109 with four), wide
    // ones for longer rows (1000 x 65536 fp32: four 107 us, three large ones 119)
    const int wide = (int)((nv + Wide::PART - 1) / Wide::PART);
    const int large = (int)((nv + Large::PART - 1) / Large::PART);
    a.cluster = std::min(large <= 2 ? large : wide, kMaxCluster);
    // few rows: more CTAs for each, down to a vector or two a thread
    while (a.cluster < kMaxCluster && a.rows * a.cluster <= num_sms() && nv > Narrow::NT * 2 * a.cluster)
      a.cluster = std::min(2 * a.cluster, kMaxCluster);
    a.part_vecs = (int)((nv + a.cluster - 1) / a.cluster);
    if (a.part_vecs <= Narrow::PART && a.k <= Narrow::MAXK) e = launch_sized<DT, Narrow>(a, s);
    else if (a.part_vecs <= Wide::PART && a.k <= Wide::MAXK) e = launch_sized<DT, Wide>(a, s);
    else if (a.k <= Large::MAXK) e = launch_sized<DT, Large>(a, s);
    else e = launch_sized<DT, Deep>(a, s);
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
