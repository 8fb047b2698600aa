// Norms of the workers' gradients over many tensors, and their clipping
// (scape_grad_norm, scape_clip_grads).
//
// A worker's tensors are cut into chunks.  norm_chunks adds up the squares of a
// chunk (fp32 over 64 elements of a thread, scaled where they leave its range; 64 bits from
// there on) and leaves one partial sum a chunk; norm_finish adds up a worker's partials in a fixed order;
// clip_chunks multiplies.  The scale is known only after the last element, so a
// clipped gradient is read twice: the floor is one reading, and what the second
// one finds in L2 is what can be saved of it.  clip_chunks therefore goes from the
// last chunk to the first.
//
// All three are bound by HBM: 1775 M bf16 elements of 291 tensors in 496 us (7.2 TB/s, read
// only); 558 M bf16 clipped in 520 us, where all bytes moved take 495 us at a copy's rate.
//
// The table of tensors travels in the kernels' parameters (at most 32764 bytes), so
// there is nothing to copy to the device and a captured graph keeps its own.
#include <algorithm>
#include <cmath>
#include <vector>

#include "host.cuh"
#include "objective.cuh"
#include "scape_kernels.cuh"

#define SCAPE_API extern "C" __attribute__((visibility("default")))

namespace scape {
namespace {

constexpr int kThreads = 256;
constexpr int kResident = 4;  // CTAs of an SM: 64 registers a thread, 128 KB of loads in flight
constexpr int kBatch = 8;     // vectors that a thread has in flight
constexpr uint64_t kMinChunk = 4096, kMaxChunkElems = 65536;
constexpr int kMaxGroups = kMaxW;

struct Tensor {
  const void* src;
  void* dst;
  uint64_t n;
  uint32_t chunk0;  // its first chunk of this table
  uint32_t part0;   // ... of all
  uint32_t group;
};

// Tensors of one type (and one type of results).
template <int CAP>
struct Table {
  Tensor t[CAP];
  int n;
  uint32_t chunks;
  uint32_t chunk_elems;
};

// The tensor of chunk c: the last one that starts at or before it.
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& tb, uint32_t c) {
  int lo = 0, hi = tb.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tb.t[mid].chunk0 <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Squares of a vector's elements times "by".  (A call, so that the loop keeps its registers.)
template <int DT>
__device__ __noinline__ float squares_by(const uint4 v, float by) {
  using E = Elem<DT>;
  float f[E::kPerVec];
  E::unpack(v, f);
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < E::kPerVec; j++) s = __fmaf_rn(f[j] * by, f[j] * by, s);
  return s;
}

// Sum of squares of a thread's batch.  In fp32 it is right to 2^-18 as long as it
// is neither beyond fp32's range nor so small that squares were lost below it;
// otherwise the batch is added up again, scaled by a power of two: elements of at most
// 2^-40 times 2^100 (the least one becomes 2^-49), others times 2^-70 (the largest one becomes
// 2^58, and what is lost below 2^-63 does not count beside it).  Zeros go that way, too, -0
// among them.  2^28 bf16 elements that are all -0, or 1e-20, or 1e30: 104 us, random ones 93.
// (Added up in 64 bits, of which this GPU does few: 1571.)
template <int DT>
__device__ __forceinline__ double squares(const uint4 (&v)[kBatch]) {
  using E = Elem<DT>;
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kBatch; i++) {
    float f[E::kPerVec];
    E::unpack(v[i], f);
#pragma unroll
    for (int j = 0; j < E::kPerVec; j++) s[j & 1] = __fmaf_rn(f[j], f[j], s[j & 1]);
  }
  const float sum = s[0] + s[1];
  if (sum > 0x1p-80f && sum < 0x1p120f) return (double)sum;
  const bool small = sum < 1.0f;  // (not of NaN)
  float scaled = 0.0f;
#pragma unroll
  for (int i = 0; i < kBatch; i++)
    if (v[i].x | v[i].y | v[i].z | v[i].w) scaled += squares_by<DT>(v[i], small ? 0x1p100f : 0x1p-70f);
  return (double)scaled * (small ? 0x1p-200 : 0x1p140);
}

template <int DT>
__device__ double chunk_squares(const void* base, uint64_t first, uint32_t n) {
  using E = Elem<DT>;
  using T = typename E::T;
  const T* p = static_cast<const T*>(base) + first;
  const int tid = threadIdx.x;
  // elements in front of the first 16-byte boundary, whole vectors, the rest
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T);
  const uint32_t head = min(n, off ? (uint32_t)E::kPerVec - off : 0u);
  const uint32_t nv = (n - head) / E::kPerVec;
  const uint32_t done = head + nv * E::kPerVec;
  double d = 0.0;
  if (tid < head) {
    const float x = E::load(p + tid);
    d = (double)x * x;
  }
  if (done + tid < n) {  // fewer than a vector
    const float x = E::load(p + done + tid);
    d += (double)x * x;
  }
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  for (uint32_t v0 = tid; v0 < nv; v0 += kThreads * kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      const uint32_t at = v0 + i * kThreads;
      v[i] = at < nv ? ld_row_u4(q + at) : make_uint4(0, 0, 0, 0);
    }
    d += squares<DT>(v);
  }
  return d;
}

template <int CAP, int DT>
__global__ __launch_bounds__(kThreads, kResident) void norm_chunks(const __grid_constant__ Table<CAP> tb,
                                                                   double* __restrict__ part) {
  __shared__ double buf[32];
  grid_launch_dependents();
  grid_dependency_wait();
  for (uint32_t c = blockIdx.x; c < tb.chunks; c += gridDim.x) {
    const Tensor& t = tb.t[tensor_of(tb, c)];
    const uint64_t first = (uint64_t)(c - t.chunk0) * tb.chunk_elems;
    const uint32_t n = (uint32_t)min((uint64_t)tb.chunk_elems, t.n - first);
    const double d = cta_sum(chunk_squares<DT>(t.src, first, n), buf);
    if (threadIdx.x == 0) part[t.part0 + (c - t.chunk0)] = d;
  }
}

struct Groups {
  uint32_t chunk0[kMaxGroups + 1];
};

// One CTA a group.
__global__ __launch_bounds__(1024) void norm_finish(const __grid_constant__ Groups g,
                                                    const double* __restrict__ part, float max_norm,
                                                    float* __restrict__ norms,
                                                    float2* __restrict__ scales) {
  __shared__ double buf[32];
  grid_launch_dependents();
  grid_dependency_wait();
  double d = 0.0;
#pragma unroll 8
  for (uint32_t c = g.chunk0[blockIdx.x] + threadIdx.x; c < g.chunk0[blockIdx.x + 1]; c += 1024)
    d += part[c];
  d = cta_sum(d, buf);
  if (threadIdx.x == 0) {
    const double norm = sqrt(d);
    const float seen = (float)norm;
    norms[blockIdx.x] = seen;
    // (a norm that the caller sees as infinite or NaN is not applied, be it finite in 64 bits)
    const double scale = norm > (double)max_norm && seen < INFINITY ? (double)max_norm / norm : 1.0;
    // two factors: the scale itself may be below fp32's range where the products are not
    if (scales)
      scales[blockIdx.x] = scale < 0x1p-100 ? make_float2((float)(scale * 0x1p100), 0x1p-100f) : make_float2((float)scale, 1.0f);
  }
}

// A streaming store of 16 bytes: it does not push what is still to be read out of L2.
__device__ __forceinline__ void st_stream_u4(void* p, const uint4 v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Eight products, stored.
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, const float (&f)[8], float2 scale) {
  using E = Elem<DT>;
#pragma unroll
  for (int i = 0; i < 8 / E::kPerVec; i++) {
    float g[E::kPerVec];
#pragma unroll
    for (int j = 0; j < E::kPerVec; j++) g[j] = f[i * E::kPerVec + j] * scale.x * scale.y;
    st_stream_u4(p + i * E::kPerVec, E::pack(g));
  }
}

// dst = src * scale.  Whole stores of 16 bytes from the first boundary of dst on;
// loads of 16 bytes where src has its boundary there too.
template <int SDT, int DDT>
__device__ __forceinline__ void scale_chunk(const void* from, void* to, uint32_t n, float2 scale) {
  using S = Elem<SDT>;
  using D = Elem<DDT>;
  const typename S::T* src = static_cast<const typename S::T*>(from);
  typename D::T* dst = static_cast<typename D::T*>(to);
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(dst) & 15u) / sizeof(typename D::T);
  const uint32_t head = min(n, off ? (uint32_t)D::kPerVec - off : 0u);
  const uint32_t n8 = (n - head) / 8, done = head + n8 * 8;
  const uint32_t tid = threadIdx.x;
  if (tid < head) dst[tid] = D::make(S::load(src + tid) * scale.x * scale.y);
  if (done + tid < n) dst[done + tid] = D::make(S::load(src + done + tid) * scale.x * scale.y);
  src += head;
  dst += head;
  if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
    constexpr int V = 8 / S::kPerVec, U = 4 / V * 2;  // 128 bytes of a thread in flight
#pragma unroll 1
    for (uint32_t v0 = tid; v0 < n8; v0 += kThreads * U) {
      uint4 raw[U][V];
#pragma unroll
      for (int i = 0; i < U; i++)
        if (v0 + i * kThreads < n8) {
#pragma unroll
          for (int j = 0; j < V; j++)
            raw[i][j] = ld_row_u4(src + (size_t)(v0 + i * kThreads) * 8 + j * S::kPerVec);
        }
#pragma unroll
      for (int i = 0; i < U; i++)
        if (v0 + i * kThreads < n8) {
          float f[8];
#pragma unroll
          for (int j = 0; j < V; j++) {
            float g[S::kPerVec];
            S::unpack(raw[i][j], g);
#pragma unroll
            for (int e = 0; e < S::kPerVec; e++) f[j * S::kPerVec + e] = g[e];
          }
          store8<DDT>(dst + (size_t)(v0 + i * kThreads) * 8, f, scale);
        }
    }
  } else {
#pragma unroll 1
    for (uint32_t v0 = tid; v0 < n8; v0 += kThreads * 2) {
      float f[2][8];
#pragma unroll
      for (int i = 0; i < 2; i++)
        if (v0 + i * kThreads < n8) {
#pragma unroll
          for (int e = 0; e < 8; e++) f[i][e] = S::load(src + (size_t)(v0 + i * kThreads) * 8 + e);
        }
#pragma unroll
      for (int i = 0; i < 2; i++)
        if (v0 + i * kThreads < n8) store8<DDT>(dst + (size_t)(v0 + i * kThreads) * 8, f[i], scale);
    }
  }
}

// A kernel for each pair of types: all of them in one take 255 registers, one CTA an SM.
template <int CAP, int SDT, int DDT>
__global__ __launch_bounds__(kThreads, kResident) void clip_chunks(const __grid_constant__ Table<CAP> tb,
                                                                   const float2* __restrict__ scales) {
  grid_launch_dependents();
  grid_dependency_wait();
  for (uint32_t i = blockIdx.x; i < tb.chunks; i += gridDim.x) {
    const uint32_t c = tb.chunks - 1 - i;  // what was read last comes first
    const Tensor& t = tb.t[tensor_of(tb, c)];
    const float2 scale = scales[t.group];
    if (scale.x == 1.0f && scale.y == 1.0f && t.src == t.dst) continue;  // in place: nothing to change
    const uint64_t first = (uint64_t)(c - t.chunk0) * tb.chunk_elems;
    const uint32_t n = (uint32_t)min((uint64_t)tb.chunk_elems, t.n - first);
    scale_chunk<SDT, DDT>(static_cast<const typename Elem<SDT>::T*>(t.src) + first,
                          static_cast<typename Elem<DDT>::T*>(t.dst) + first, n, scale);
  }
}

// How the tensors are cut, by their sizes alone.
struct Cut {
  uint64_t chunk_elems = kMinChunk, chunks = 0;
};

int check_sizes(const scape_grads* g, Cut& cut) {
  if (!g) return fail(SCAPE_EINVAL, "grads is NULL");
  if (g->n_groups < 1 || g->n_groups > (uint32_t)kMaxGroups)
    return fail(SCAPE_EINVAL, "n_groups=%u must be in [1, %d]", g->n_groups, kMaxGroups);
  if (g->n_tensors >= (1u << 20)) return fail(SCAPE_EINVAL, "n_tensors must be < 2^20");
  if (g->n_tensors && !g->numel) return fail(SCAPE_EINVAL, "numel is NULL");
  if (g->first_tensor) {
    if (g->first_tensor[0] != 0 || g->first_tensor[g->n_groups] != g->n_tensors)
      return fail(SCAPE_EINVAL, "first_tensor must begin with 0 and end with n_tensors");
    for (uint32_t i = 0; i < g->n_groups; i++)
      if (g->first_tensor[i] > g->first_tensor[i + 1])
        return fail(SCAPE_EINVAL, "first_tensor must ascend");
  } else if (g->n_groups != 1) {
    return fail(SCAPE_EINVAL, "n_groups > 1 needs first_tensor");
  }
  uint64_t total = 0;
  for (uint32_t i = 0; i < g->n_tensors; i++) {
    if (g->numel[i] >= (1ull << 40)) return fail(SCAPE_EINVAL, "tensor %u: numel must be < 2^40", i);
    total += g->numel[i];
  }
  if (total >= (1ull << 44)) return fail(SCAPE_EINVAL, "the gradients must have < 2^44 elements");
  // chunks large enough that few partials are left, and one of them for every SM where there is enough for that
  // (4 x 2^20 elements: 10.7 us, with two 11.7, with eight 16.8; 2 x 2^24: 14.5, with eight 25.8)
  const uint64_t want = (uint64_t)num_sms();
  while (cut.chunk_elems < kMaxChunkElems && total / (2 * cut.chunk_elems) >= want) cut.chunk_elems *= 2;
  for (uint32_t i = 0; i < g->n_tensors; i++)
    cut.chunks += (g->numel[i] + cut.chunk_elems - 1) / cut.chunk_elems;
  if (cut.chunks >= (1ull << 31)) return fail(SCAPE_EINVAL, "too many elements or tensors");
  return SCAPE_OK;
}

int check_tensors(const scape_grads* g) {
  if (g->n_tensors && (!g->grads || !g->dtypes)) return fail(SCAPE_EINVAL, "grads and dtypes are required");
  for (uint32_t i = 0; i < g->n_tensors; i++) {
    if (!known(g->dtypes[i])) return fail(SCAPE_EINVAL, "tensor %u: unknown dtype %d", i, g->dtypes[i]);
    if (g->numel[i] && !g->grads[i]) return fail(SCAPE_EINVAL, "tensor %u is NULL", i);
    if (reinterpret_cast<uintptr_t>(g->grads[i]) % size_of(g->dtypes[i]))
      return fail(SCAPE_EINVAL, "tensor %u is not aligned to its element size", i);
  }
  return SCAPE_OK;
}

// No element is written twice, nor read after another tensor's was written over it.
int check_overlap(const scape_grads* g, void* const* out, const uint8_t* odt) {
  struct Span {
    uintptr_t a, b;
    uint32_t i;
  };
  std::vector<Span> w;
  w.reserve(g->n_tensors);
  for (uint32_t i = 0; i < g->n_tensors; i++)
    if (g->numel[i]) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(out[i]);
      w.push_back({a, a + g->numel[i] * size_of(odt[i]), i});
    }
  if (!std::is_sorted(w.begin(), w.end(), [](const Span& x, const Span& y) { return x.a < y.a; }))
    std::sort(w.begin(), w.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
  for (size_t j = 1; j < w.size(); j++)
    if (w[j].a < w[j - 1].b)
      return fail(SCAPE_EINVAL, "the results of tensors %u and %u overlap", w[j - 1].i, w[j].i);
  for (uint32_t i = 0; i < g->n_tensors; i++) {
    if (!g->numel[i]) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(g->grads[i]), b = a + g->numel[i] * size_of(g->dtypes[i]);
    size_t lo = 0, hi = w.size();  // the first span that ends behind a
    while (lo < hi) {
      const size_t mid = (lo + hi) / 2;
      if (w[mid].b > a) hi = mid;
      else lo = mid + 1;
    }
    if (lo < w.size() && w[lo].a < b &&
        !(w[lo].i == i && w[lo].a == a && odt[i] == g->dtypes[i]))
      return fail(SCAPE_EINVAL, "the result of tensor %u overlaps tensor %u", w[lo].i, i);
  }
  return SCAPE_OK;
}

// What launch_tables goes through: the tensors, and where the results go (clipping).
struct Todo {
  const scape_grads* g;
  uint32_t chunk_elems;
  const uint32_t* part0;  // of every tensor
  const uint32_t* group;
  void* const* out;
  const uint8_t* out_dtypes;
  double* part;
  const float2* scales;
  uint32_t chunks_of(uint32_t i) const { return (uint32_t)((g->numel[i] + chunk_elems - 1) / chunk_elems); }
};

// The tensors that "list" names into one table, and its launch.
template <int CAP, int SDT, int DDT>
cudaError_t launch_table(const Todo& q, const std::vector<uint32_t>& list, size_t i0, size_t i1,
                         cudaStream_t s) {
  Table<CAP> tb;
  tb.n = (int)(i1 - i0);
  tb.chunk_elems = q.chunk_elems;
  tb.chunks = 0;
  for (size_t j = i0; j < i1; j++) {
    const uint32_t i = list[j];
    tb.t[j - i0] = {q.g->grads[i], q.out ? q.out[i] : nullptr, q.g->numel[i], tb.chunks, q.part0[i], q.group[i]};
    tb.chunks += q.chunks_of(i);
  }
  const unsigned grid = std::min<unsigned>(tb.chunks, (unsigned)(kResident * num_sms()));
  if (q.out) return launch_behind(clip_chunks<CAP, SDT, DDT>, grid, kThreads, s, tb, q.scales);
  if constexpr (DDT == SCAPE_BF16) return launch_behind(norm_chunks<CAP, SDT>, grid, kThreads, s, tb, q.part);
  return cudaSuccess;
}

// All tensors of one type (and one type of results): as many tables as they need, small
// parameters for small calls.
constexpr int kSmallTable = 16, kLargeTable = 600;
template <int SDT, int DDT>
cudaError_t launch_tables(const Todo& q, cudaStream_t s) {
  std::vector<uint32_t> list;
  for (uint32_t i = 0; i < q.g->n_tensors; i++)
    if (q.g->numel[i] && q.g->dtypes[i] == SDT && (!q.out || q.out_dtypes[i] == DDT)) list.push_back(i);
  for (size_t i0 = 0; i0 < list.size(); i0 += kLargeTable) {
    const size_t i1 = std::min(list.size(), i0 + kLargeTable);
    const cudaError_t e = i1 - i0 <= (size_t)kSmallTable ? launch_table<kSmallTable, SDT, DDT>(q, list, i0, i1, s)
                                                         : launch_table<kLargeTable, SDT, DDT>(q, list, i0, i1, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int SDT>
cudaError_t launch_from(const Todo& q, cudaStream_t s) {
  cudaError_t e = launch_tables<SDT, SCAPE_BF16>(q, s);
  if (e == cudaSuccess && q.out) e = launch_tables<SDT, SCAPE_F16>(q, s);
  if (e == cudaSuccess && q.out) e = launch_tables<SDT, SCAPE_F32>(q, s);
  return e;
}
cudaError_t launch_all(const Todo& q, cudaStream_t s) {
  cudaError_t e = launch_from<SCAPE_BF16>(q, s);
  if (e == cudaSuccess) e = launch_from<SCAPE_F16>(q, s);
  if (e == cudaSuccess) e = launch_from<SCAPE_F32>(q, s);
  return e;
}

uint64_t bytes_of(const Cut& cut) { return cut.chunks * 8 + kMaxGroups * 8; }

int norm_and_clip(const scape_grads* g, bool clip, float max_norm, void* const* out, const uint8_t* odt,
                  float* norms, void* workspace, uint64_t workspace_bytes, void* stream) {
  Cut cut;
  if (int rc = check_sizes(g, cut)) return rc;
  if (int rc = check_tensors(g)) return rc;
  if (clip) {
    if (!(max_norm > 0.0f)) return fail(SCAPE_EINVAL, "max_norm must be > 0");
    if (!out) {
      out = const_cast<void* const*>(reinterpret_cast<const void* const*>(g->grads));
      odt = g->dtypes;
    } else {
      if (g->n_tensors && !odt) return fail(SCAPE_EINVAL, "out_dtypes is NULL");
      for (uint32_t i = 0; i < g->n_tensors; i++) {
        if (!known(odt[i])) return fail(SCAPE_EINVAL, "out %u: unknown dtype %d", i, odt[i]);
        if (g->numel[i] && !out[i]) return fail(SCAPE_EINVAL, "out %u is NULL", i);
        if (reinterpret_cast<uintptr_t>(out[i]) % size_of(odt[i]))
          return fail(SCAPE_EINVAL, "out %u is not aligned to its element size", i);
      }
    }
    if (int rc = check_overlap(g, out, odt)) return rc;
  }
  if (!norms || reinterpret_cast<uintptr_t>(norms) % 4)
    return fail(SCAPE_EINVAL, "norms is required, aligned to its element size");
  const uint64_t need = bytes_of(cut);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < need)
    return fail(SCAPE_EINVAL, "workspace must be %llu bytes, 16-byte aligned", (unsigned long long)need);

  double* part = static_cast<double*>(workspace);
  float2* scales = reinterpret_cast<float2*>(part + cut.chunks);
  std::vector<uint32_t> group(g->n_tensors), part0(g->n_tensors);
  Todo q{g, (uint32_t)cut.chunk_elems, part0.data(), group.data(), nullptr, nullptr, part, scales};
  Groups gr{};
  uint32_t at = 0;
  for (uint32_t w = 0, i = 0; w < g->n_groups; w++) {
    gr.chunk0[w] = at;
    const uint32_t end = g->first_tensor ? (uint32_t)g->first_tensor[w + 1] : g->n_tensors;
    for (; i < end; i++) {
      group[i] = w;
      part0[i] = at;
      at += q.chunks_of(i);
    }
    gr.chunk0[w + 1] = at;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_all(q, s);
  if (e != cudaSuccess) return fail(SCAPE_ECUDA, "norm_chunks: %s", cudaGetErrorString(e));
  e = launch_behind(norm_finish, g->n_groups, 1024, s, gr, (const double*)part, max_norm, norms,
                    clip ? scales : (float2*)nullptr);
  if (e != cudaSuccess) return fail(SCAPE_ECUDA, "norm_finish: %s", cudaGetErrorString(e));
  if (!clip) return SCAPE_OK;
  q.out = out;
  q.out_dtypes = odt;
  e = launch_all(q, s);
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "clip_chunks: %s", cudaGetErrorString(e));
}

}  // namespace
}  // namespace scape

SCAPE_API int scape_grad_workspace(const scape_grads* grads, uint64_t* bytes) {
  using namespace scape;
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  *bytes = 0;
  Cut cut;
  if (int rc = check_sizes(grads, cut)) return rc;
  *bytes = bytes_of(cut);
  return SCAPE_OK;
}

SCAPE_API int scape_grad_norm(const scape_grads* grads, float* norms, void* workspace,
                              uint64_t workspace_bytes, void* stream) {
  try {
    return scape::norm_and_clip(grads, false, 0.0f, nullptr, nullptr, norms, workspace, workspace_bytes, stream);
  } catch (...) {
    return scape::fail(SCAPE_ENOMEM, "host allocation failed");
  }
}

SCAPE_API int scape_clip_grads(const scape_grads* grads, float max_norm, void* const* out,
                               const uint8_t* out_dtypes, float* norms, void* workspace,
                               uint64_t workspace_bytes, void* stream) {
  try {
    return scape::norm_and_clip(grads, true, max_norm, out, out_dtypes, norms, workspace, workspace_bytes, stream);
  } catch (...) {
    return scape::fail(SCAPE_ENOMEM, "host allocation failed");
  }
}
