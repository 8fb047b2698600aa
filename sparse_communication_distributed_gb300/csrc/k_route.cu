// Expert routing: top-k experts of every token, their weights, how many
// choices every expert of every group of tokens got, the balance loss and the z
// loss; and the gradient of the logits.
//
// Forward.  A token's logits lie across L lanes of a warp (L a power of two, 8
// columns a lane, more for over 256 experts).  The tokens are cut into chunks,
// one CTA each; within a chunk the CTA goes group by group and leaves, for every
// group that the chunk touches, the sums of p and the counts over its tokens in
// a slot of the workspace.  Chunk i and group g use slot i + g: along the
// tokens either i or g moves on, so no two pairs share a slot and a group's
// slots are adjacent.  A second kernel adds a group's slots up in order, so the
// sums do not depend on the schedule.
//
// Backward.  With d_e = dB / G' * E c_ge / (k T_g^2) of the token's group,
//   d x_j = p_j (d_j - sum_e p_e d_e) + (2 dZ / T) lse p_j + (weights' part),
// where the weights' part is w_i (dw_i - sum w dw) at the chosen experts if
// renormalised, else p_j (dw_j [chosen] - sum w dw).
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
  int E, k, L, renorm;  // L: lanes of a token
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

// First group whose end lies beyond token t (a.G if none).
__device__ __forceinline__ int64_t group_at(const RouteArgs& a, int64_t t) {
  int64_t lo = 0, hi = a.G;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (bound_of(a, mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

template <class F>
__device__ __forceinline__ float lanes_reduce(float x, int L, F f) {
  for (int o = L >> 1; o; o >>= 1) x = f(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
__device__ __forceinline__ float lanes_sum(float x, int L) {
  return lanes_reduce(x, L, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float lanes_max(float x, int L) {
  return lanes_reduce(x, L, [](float a, float b) { return fmaxf(a, b); });
}

// The columns of a lane: column 8 (c L + sub) + j is its value 8 c + j.
template <int VPL>
__device__ __forceinline__ int col_of(int L, int sub, int j) {
  return ((j >> 3) * L + sub) * 8 + (j & 7);
}

// A lane's logits of token t, -inf beyond the experts.
template <int DT, int VPL, bool VEC>
__device__ __forceinline__ void load_row(const void* base, int64_t t, int64_t stride, int Ex, int L,
                                         int sub, bool in, float (&x)[VPL]) {
  using E = Elem<DT>;
  const typename E::T* p = static_cast<const typename E::T*>(base) + t * stride;
#pragma unroll
  for (int c = 0; c < VPL / 8; c++) {
    const int col = (c * L + sub) * 8;
    if (VEC) {
      constexpr int N = 8 / E::kPerVec;
#pragma unroll
      for (int h = 0; h < N; h++) {
        float f[E::kPerVec];
        const uint4 ninf = make_uint4(E::kNegInf2, E::kNegInf2, E::kNegInf2, E::kNegInf2);
        E::unpack(in && col < Ex ? ld_row_u4(p + col + h * E::kPerVec) : ninf, f);
#pragma unroll
        for (int j = 0; j < E::kPerVec; j++) x[c * 8 + h * E::kPerVec + j] = f[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) x[c * 8 + j] = in && col + j < Ex ? E::load(p + col + j) : neg_inf();
    }
  }
}

template <int DT, int VPL, bool VEC>
__global__ __launch_bounds__(kThreads) void route_chunks(const RouteArgs a) {
  extern __shared__ unsigned char smem[];
  const int L = a.L, per_warp = 32 / L;
  float* sp = reinterpret_cast<float*>(smem);                   // kWarps x E
  int32_t* sc = reinterpret_cast<int32_t*>(sp + kWarps * a.E);  // E
  float* sw = reinterpret_cast<float*>(sc + a.E);               // tokens of a round x k
  int32_t* si = reinterpret_cast<int32_t*>(sw + kWarps * per_warp * a.k);
  __shared__ float fbuf[32];
  __shared__ int32_t ibuf[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int sub = lane & (L - 1), slot = lane / L;
  const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  if (blockIdx.x == 0 && tid == 0) *a.done = 0;

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
    float acc[VPL];
#pragma unroll
    for (int j = 0; j < VPL; j++) acc[j] = 0.0f;
    float zsum = 0.0f;
    int32_t nlive = 0;
    for (int i = tid; i < a.E; i += kThreads) sc[i] = 0;
    __syncthreads();
    for (int64_t r = at; r < end; r += kWarps * per_warp) {
      const int64_t t = r + wid * per_warp + slot;
      const bool in = t < end;
      float x[VPL];
      load_row<DT, VPL, VEC>(a.x, t, a.stride, a.E, L, sub, in, x);
      bool ok = in && inside && (!a.valid || a.valid[t] != 0);
      float m = neg_inf();
      bool nan = false;
#pragma unroll
      for (int j = 0; j < VPL; j++) {
        m = fmaxf(m, x[j]);
        nan |= x[j] != x[j];
      }
      m = lanes_max(m, L);
      nan = lanes_max(nan ? 1.0f : 0.0f, L) != 0.0f;
      ok = ok && (m > neg_inf() || nan);
      const float sh = shift_of(m);
      float p[VPL], s = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; j++) {
        p[j] = ex2((x[j] - sh) * kLog2e);
        s += p[j];
      }
      s = lanes_sum(s, L);
      const float lse = sh + logf(s), inv = 1.0f / s;
      if (ok) {
#pragma unroll
        for (int j = 0; j < VPL; j++) acc[j] += p[j] * inv;
        if (sub == 0) {
          zsum += lse * lse;
          nlive++;
        }
      }
      // the k best, one after the other
      uint32_t key[VPL];
#pragma unroll
      for (int j = 0; j < VPL; j++)
        key[j] = col_of<VPL>(L, sub, j) < a.E ? order_key(x[j]) : 0u;
      const int base = (wid * per_warp + slot) * a.k;
      float sel = 0.0f, top = 0.0f;
      for (int i = 0; i < a.k; i++) {
        uint64_t best = 0;
#pragma unroll
        for (int j = 0; j < VPL; j++) {
          const uint64_t v = (uint64_t)key[j] << 32 | (uint32_t)~col_of<VPL>(L, sub, j);
          best = v > best && key[j] ? v : best;
        }
        for (int o = L >> 1; o; o >>= 1) {
          const uint64_t other = __shfl_xor_sync(kFull, best, o);
          best = other > best ? other : best;
        }
        const int col = (int)~(uint32_t)best;
        const uint32_t kb = (uint32_t)(best >> 32);
        const float v = kb == 0xFFFFFFFFu ? __uint_as_float(0x7FFFFFFFu)
                        : __uint_as_float((kb & 0x80000000u) ? kb & 0x7FFFFFFFu : ~kb);
#pragma unroll
        for (int j = 0; j < VPL; j++)
          if (col_of<VPL>(L, sub, j) == col) key[j] = 0;
        if (i == 0) top = shift_of(v);
        const float e = a.renorm ? ex2((v - top) * kLog2e) : ex2((v - sh) * kLog2e) * inv;
        sel += e;
        if (sub == 0) {
          sw[base + i] = e;
          si[base + i] = ok ? col : -1;
          if (ok) atomicAdd(&sc[col], 1);
        }
      }
      __syncwarp();
      const float scale = a.renorm ? 1.0f / sel : 1.0f;
      const int64_t left = end - (r + wid * per_warp);
      const int n = (int)(left < per_warp ? left : per_warp) * a.k;
      // one value of the token's scale for each lane that writes it
      for (int i = 0; i < per_warp * a.k; i += 32) {
        const int q = i + lane, tok = q < per_warp * a.k ? q / a.k : 0;
        const float sc_ = __shfl_sync(kFull, scale, tok * L);
        if (q < n) {
          const int32_t e = si[wid * per_warp * a.k + q];
          const int64_t o = (r + wid * per_warp) * a.k + q;
          a.idx[o] = e;
          a.weights[o] = e < 0 ? 0.0f : sw[wid * per_warp * a.k + q] * sc_;
        }
      }
      __syncwarp();
    }
    if (inside) {  // the slot of this chunk and group
#pragma unroll
      for (int j = 0; j < VPL; j++) {
        for (int o = L; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(kFull, acc[j], o);
        const int col = col_of<VPL>(L, sub, j);
        if (slot == 0 && col < a.E) sp[wid * a.E + col] = acc[j];
      }
      const float z = cta_sum(zsum, fbuf);
      const int32_t n = cta_sum(nlive, ibuf);
      __syncthreads();
      const int64_t sl = blockIdx.x + g;
      for (int i = tid; i < a.E; i += kThreads) {
        float p = 0.0f;
        for (int w = 0; w < kWarps; w++) p += sp[w * a.E + i];
        a.part_p[sl * a.E + i] = p;
        a.part_c[sl * a.E + i] = sc[i];
      }
      if (tid == 0) {
        a.part_n[sl] = n;
        a.part_z[sl] = z;
      }
    }
    __syncthreads();
    if (g < a.G && bound_of(a, g + 1) <= end) g++;
    at = end;
  }
}

// One CTA per group and block of kThreads / 8 columns; 8 threads share a
// column's slots.  The last CTA to finish adds up what the groups contribute.
constexpr int kCols = kThreads / 8;

__global__ __launch_bounds__(kThreads) void route_finish(const RouteArgs a) {
  __shared__ float fbuf[32];
  __shared__ int32_t ibuf[32];
  __shared__ bool last;
  const int tid = threadIdx.x;
  const int64_t g = blockIdx.x;
  const int nb = gridDim.y;
  const int64_t lo = bound_of(a, g), hi = bound_of(a, g + 1);
  const int64_t s0 = lo / a.chunk + g, s1 = hi > lo ? (hi - 1) / a.chunk + g + 1 : s0;
  int32_t n = 0;
  for (int64_t s = s0 + tid; s < s1; s += kThreads) n += a.part_n[s];
  n = cta_sum(n, ibuf);
  const int col = blockIdx.y * kCols + (tid >> 3);
  float p = 0.0f;
  int32_t c = 0;
  if (col < a.E)
    for (int64_t s = s0 + (tid & 7); s < s1; s += 8) {
      p += a.part_p[s * a.E + col];
      c += a.part_c[s * a.E + col];
    }
  for (int o = 4; o; o >>= 1) {
    p += __shfl_xor_sync(kFull, p, o);
    c += __shfl_xor_sync(kFull, c, o);
  }
  if (col < a.E && (tid & 7) == 0) a.counts[g * a.E + col] = c;
  const float tg = (float)max(n, 1);
  const float b = (tid & 7) == 0 && col < a.E ? p * (float)c : 0.0f;
  const float bal = cta_sum(b, fbuf) * ((float)a.E / ((float)a.k * tg)) / tg;
  if (tid == 0) {
    a.part_b[g * nb + blockIdx.y] = bal;
    if (blockIdx.y == 0) a.live[g] = n;
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
    const int64_t lo2 = bound_of(a, i), hi2 = bound_of(a, i + 1);
    if (hi2 > lo2)
      for (int64_t s = lo2 / a.chunk + i; s <= (hi2 - 1) / a.chunk + i; s++) z += a.part_z[s];
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

template <int DT, int VPL, bool VEC>
__global__ __launch_bounds__(kThreads) void route_grad(const RouteArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  const int L = a.L, per_warp = 32 / L;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int sub = lane & (L - 1), slot = lane / L;
  const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  const float dB = a.dl ? a.dl[0] : 0.0f, dZ = a.dl ? a.dl[1] : 0.0f;
  const float zc = 2.0f * dZ / (float)max(a.blive[a.G], 1);
  const float bc = dB / (float)max(a.blive[a.G + 1], 1) * ((float)a.E / (float)a.k);
  for (int64_t r = t0; r < t1; r += kWarps * per_warp) {
    const int64_t t = r + wid * per_warp + slot;
    const bool in = t < t1;
    float x[VPL], y[VPL];
    load_row<DT, VPL, VEC>(a.x, t, a.stride, a.E, L, sub, in, x);
    const bool ok = in && a.bidx[t * a.k] >= 0;
    const int64_t g = in ? group_at(a, t) : 0;
    float m = neg_inf();
#pragma unroll
    for (int j = 0; j < VPL; j++) m = fmaxf(m, x[j]);
    m = shift_of(lanes_max(m, L));
    float s = 0.0f, pd = 0.0f;
    float tg = 1.0f;
    if (ok && g < a.G) tg = (float)max(a.blive[g], 1);
    const float coef = bc / tg / tg;
#pragma unroll
    for (int j = 0; j < VPL; j++) {
      const int col = col_of<VPL>(L, sub, j);
      x[j] = ex2((x[j] - m) * kLog2e);
      s += x[j];
      y[j] = ok && g < a.G && col < a.E ? coef * (float)a.bcounts[g * a.E + col] : 0.0f;
      pd += x[j] * y[j];
    }
    s = lanes_sum(s, L);
    pd = lanes_sum(pd, L);
    const float inv = 1.0f / s, lse = m + logf(s);
    pd = pd * inv - zc * lse;
    // the chosen experts: their weights, and what the weights' gradients give
    float top = m, den = s, dot = 0.0f;
    if (ok && a.dw) {
      if (a.renorm) {
        top = Elem<DT>::load(static_cast<const T*>(a.x) + t * a.stride + min(a.bidx[t * a.k], a.E - 1));
        top = shift_of(top);
        den = 0.0f;
        for (int i = 0; i < a.k; i++) {
          const int e = min(max(a.bidx[t * a.k + i], 0), a.E - 1);
          den += ex2((Elem<DT>::load(static_cast<const T*>(a.x) + t * a.stride + e) - top) * kLog2e);
        }
      }
      for (int i = 0; i < a.k; i++) {
        const int e = min(max(a.bidx[t * a.k + i], 0), a.E - 1);
        const float v = Elem<DT>::load(static_cast<const T*>(a.x) + t * a.stride + e);
        dot += ex2((v - top) * kLog2e) / den * a.dw[t * a.k + i];
      }
    }
    if (!a.renorm) pd += dot;
#pragma unroll
    for (int j = 0; j < VPL; j++) y[j] = x[j] * inv * (y[j] - pd);
    if (ok && a.dw)
      for (int i = 0; i < a.k; i++) {
        const int e = a.bidx[t * a.k + i];
        const float d = a.dw[t * a.k + i] - (a.renorm ? dot : 0.0f);
#pragma unroll
        for (int j = 0; j < VPL; j++)
          if (col_of<VPL>(L, sub, j) == e) {
            const float v = Elem<DT>::load(static_cast<const T*>(a.x) + t * a.stride + e);
            y[j] += ex2((v - top) * kLog2e) / den * d;
          }
      }
    if (!in) continue;
    T* gp = static_cast<T*>(a.grad) + t * a.gstride;
#pragma unroll
    for (int j = 0; j < VPL; j++) {
      const int col = col_of<VPL>(L, sub, j);
      if (col < a.E) gp[col] = E::make(ok ? y[j] : 0.0f);
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

// Tokens of a chunk: the chunks fill the GPU twice over, in whole rounds of a
// CTA's tokens.
uint64_t chunk_of(const scape_route_args* q) {
  const uint64_t want = (q->tokens + 303) / 304;
  return (want + 255) / 256 * 256 ? (want + 255) / 256 * 256 : 256;
}

struct Workspace {
  uint64_t slots, nb, part_p, part_c, part_n, part_z, part_b, done, bytes;
};

Workspace workspace_of(const scape_route_args* q) {
  Workspace w{};
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
  const int vpl = q->experts <= 256 ? 8 : q->experts <= 512 ? 16 : 32;
  a.L = 1;
  while (a.L * vpl < q->experts) a.L <<= 1;
}

template <int DT, int VPL, bool VEC>
void launch(const RouteArgs& a, unsigned grid, bool back, cudaStream_t s) {
  if (back) {
    route_grad<DT, VPL, VEC><<<grid, kThreads, 0, s>>>(a);
  } else {
    const size_t sm =  // under 48 KB at every size
        (size_t)(kWarps + 1) * a.E * 4 + (size_t)kWarps * (32 / a.L) * a.k * 8;
    route_chunks<DT, VPL, VEC><<<grid, kThreads, sm, s>>>(a);
  }
}

template <int DT>
void launch_dt(const RouteArgs& a, bool vec, unsigned grid, bool back, cudaStream_t s) {
  if (a.E <= 256) {
    if (vec) launch<DT, 8, true>(a, grid, back, s);
    else launch<DT, 8, false>(a, grid, back, s);
  } else if (a.E <= 512) {
    launch<DT, 16, false>(a, grid, back, s);
  } else {
    launch<DT, 32, false>(a, grid, back, s);
  }
}

void launch_any(int dtype, const RouteArgs& a, bool vec, unsigned grid, bool back, cudaStream_t s) {
  if (dtype == SCAPE_BF16) launch_dt<SCAPE_BF16>(a, vec, grid, back, s);
  else if (dtype == SCAPE_F16) launch_dt<SCAPE_F16>(a, vec, grid, back, s);
  else launch_dt<SCAPE_F32>(a, vec, grid, back, s);
}

// 16-byte loads need every row on a 16-byte boundary and whole vectors of 8.
bool vec_ok(const scape_route_args* q) {
  const uint64_t es = q->dtype == SCAPE_F32 ? 4 : 2;
  return !misaligned(q->logits, 16) && q->row_stride * es % 16 == 0 && q->experts % 8 == 0;
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
  if (!workspace || misaligned(workspace, 16) || workspace_bytes < w.bytes)
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
  a.done = reinterpret_cast<uint32_t*>(ws + w.done);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)((args->tokens + a.chunk - 1) / a.chunk);
  launch_any(args->dtype, a, vec_ok(args), grid ? grid : 1u, false, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SCAPE_ECUDA, "route_chunks: %s", cudaGetErrorString(e));
  route_finish<<<dim3((unsigned)args->n_groups, (unsigned)w.nb), kThreads, 0, s>>>(a);
  e = cudaGetLastError();
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
  const unsigned grid = (unsigned)((args->tokens + a.chunk - 1) / a.chunk);
  launch_any(args->dtype, a, vec_ok(args), grid, true, static_cast<cudaStream_t>(stream));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "route_grad: %s", cudaGetErrorString(e));
}
