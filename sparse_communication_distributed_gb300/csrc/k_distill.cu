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
  a.tau = q.temperature;
  a.c = kLog2e / q.temperature;
  a.kd = q.kd_weight;
  a.ce = q.ce_weight;
  const uint64_t cap = (uint64_t)num_sms() * 4;
  const unsigned grid = (unsigned)(q.rows < cap ? q.rows : cap);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (q.dtype == SCAPE_BF16) distill_rows<SCAPE_BF16><<<grid, kThreads, 0, s>>>(a);
  else if (q.dtype == SCAPE_F16) distill_rows<SCAPE_F16><<<grid, kThreads, 0, s>>>(a);
  else distill_rows<SCAPE_F32><<<grid, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "distill_rows: %s", cudaGetErrorString(e));
}
