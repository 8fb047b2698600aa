// Tokens sorted by expert and back (scape_expert_plan, _dispatch, _combine,
// _combine_backward).
//
// The plan is a stable counting sort of the tokens x k choices: place_counts counts
// the experts of every chunk of choices, place_scan turns the counts into each
// chunk's first place in every expert's segment, place_choices ranks the choices
// inside a chunk (a warp's 32 at a time, equal experts found with match.any) and
// writes both directions of the permutation.  Up to one chunk of choices all of it
// is one kernel of one CTA.  (A place_choices that adds up the counts itself saves a
// kernel and gains nothing: 7.4 us either way for 48 chunks, 12.1 instead of 7.8 for 64 and
// 256 experts.)
//
// Rows move in 16-byte vectors where their length and addresses allow, else in
// units of 4 or 2 bytes.  A token's row is read once and stored to its k places
// (dispatch), or its k rows are summed in registers (combine): HBM sees each row
// once.
#include <algorithm>

#include "host.cuh"
#include "objective.cuh"
#include "scape_kernels.cuh"

#define SCAPE_API extern "C" __attribute__((visibility("default")))

namespace scape {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRounds = 8;                          // choices of a thread
constexpr int kChunk = kThreads * kRounds;          // choices of a CTA
constexpr int kMaxExperts = 1024, kMaxChoices = 32;

struct PlanArgs {
  const int32_t* idx;
  int64_t n;  // choices
  int E;
  int align;
  int64_t chunks, capacity;
  int32_t* offsets;
  int32_t* slots;
  int32_t* source;
  uint32_t* bad;
  int32_t* counts;  // chunks x E: choices; after place_scan their exclusive sums over the chunks
  int32_t* totals;  // E
};

// The expert of a choice, -1 for none.
__device__ __forceinline__ int expert_of(const PlanArgs& a, int64_t i) {
  if (i >= a.n) return -1;
  const int e = a.idx[i];
  return e < a.E ? e : -1;
}

__global__ __launch_bounds__(kThreads) void place_counts(const PlanArgs a) {
  __shared__ int32_t h[kMaxExperts];
  for (int e = threadIdx.x; e < a.E; e += kThreads) h[e] = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();  // (not before: place_choices reads idx ahead of its own wait)
  const int64_t base = (int64_t)blockIdx.x * kChunk;
#pragma unroll
  for (int r = 0; r < kRounds; r++) {
    const int e = expert_of(a, base + r * kThreads + threadIdx.x);
    if (e >= 0) atomicAdd(&h[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = h[e];
}

// 32 experts a CTA, the chunks in 32 slices.
__global__ __launch_bounds__(1024) void place_scan(const PlanArgs a) {
  __shared__ int32_t sums[32][33];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  const int64_t per = (a.chunks + 31) / 32;
  const int64_t b0 = min(a.chunks, slice * per), b1 = min(a.chunks, b0 + per);
  int32_t s = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int64_t b = b0; b < b1; b++) s += a.counts[b * a.E + e];
  }
  sums[slice][lane] = s;
  __syncthreads();
  const int32_t mine = sums[lane][slice];  // (expert "slice", slice "lane")
  const int32_t incl = (int32_t)warp_incl_scan((uint32_t)mine, lane);
  __syncthreads();
  sums[lane][slice] = incl - mine;
  if (lane == 31 && blockIdx.x * 32 + slice < a.E) a.totals[blockIdx.x * 32 + slice] = incl;
  __syncthreads();
  if (e < a.E) {
    int32_t run = sums[slice][lane];
#pragma unroll 8
    for (int64_t b = b0; b < b1; b++) {
      const int32_t c = a.counts[b * a.E + e];
      a.counts[b * a.E + e] = run;
      run += c;
    }
  }
}

// SINGLE: one chunk, whose own counts are the totals.
template <bool SINGLE>
__global__ __launch_bounds__(kThreads) void place_choices(const PlanArgs a) {
  __shared__ uint16_t hist[kWarps][kMaxExperts];  // a warp's choices of each expert, then those of the warps before it
  __shared__ int32_t base[kMaxExperts];           // place of the chunk's first choice of each expert
  __shared__ int32_t start[kMaxExperts + 1];      // segments
  __shared__ int32_t total[kMaxExperts];
  __shared__ uint32_t scan[kWarps + 1];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  grid_launch_dependents();
  for (int i = tid; i < kWarps * kMaxExperts / 2; i += kThreads) reinterpret_cast<uint32_t*>(hist)[i] = 0;
  __syncthreads();
  // (idx was complete before place_counts let this kernel start)
  if (SINGLE) grid_dependency_wait();
  // a warp's choices follow one another: 32 a round
  const int64_t first = (int64_t)blockIdx.x * kChunk + wid * (32 * kRounds) + lane;
  int ex[kRounds];
  uint32_t rank[kRounds];
  uint32_t n_bad = 0;
#pragma unroll
  for (int r = 0; r < kRounds; r++) {
    const int64_t i = first + r * 32;
    ex[r] = -1;
    if (i < a.n) {
      const int e = a.idx[i];
      n_bad += e >= a.E;
      ex[r] = e >= 0 && e < a.E ? e : -1;
    }
  }
#pragma unroll
  for (int r = 0; r < kRounds; r++) {
    const uint32_t same = __match_any_sync(kFull, ex[r]);
    const int leader = __ffs(same) - 1;
    rank[r] = 0;
    if (ex[r] >= 0) rank[r] = hist[wid][ex[r]] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (ex[r] >= 0 && lane == leader) hist[wid][ex[r]] += (uint16_t)__popc(same);
    __syncwarp();
  }
  if (a.bad) {
    n_bad = __reduce_add_sync(kFull, n_bad);
    if (lane == 0 && n_bad) atomicAdd(a.bad, n_bad);
  }
  __syncthreads();
  if (!SINGLE) grid_dependency_wait();
  // segments: each thread has a run of experts
  const int per = (a.E + kThreads - 1) / kThreads;
  uint32_t room = 0;
  for (int j = 0; j < per; j++) {
    const int e = tid * per + j;
    if (e < a.E) {
      uint32_t own = 0;
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        const uint32_t c = hist[w][e];
        hist[w][e] = (uint16_t)own;
        own += c;
      }
      total[e] = SINGLE ? (int32_t)own : a.totals[e];
      base[e] = SINGLE ? 0 : a.counts[(int64_t)blockIdx.x * a.E + e];
      room += (uint32_t)((total[e] + a.align - 1) / a.align * a.align);
    }
  }
  uint32_t all;
  uint32_t at = block_incl_scan<kThreads>(room, scan, &all) - room;
  for (int j = 0; j < per; j++) {
    const int e = tid * per + j;
    if (e < a.E) {
      start[e] = (int32_t)at;
      base[e] += (int32_t)at;
      at += (uint32_t)((total[e] + a.align - 1) / a.align * a.align);
    }
  }
  if (tid == 0) start[a.E] = (int32_t)all;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; r++) {
    const int64_t i = first + r * 32;
    if (i >= a.n) break;
    int32_t slot = -1;
    if (ex[r] >= 0) {
      slot = base[ex[r]] + hist[wid][ex[r]] + (int32_t)rank[r];
      a.source[slot] = (int32_t)i;
    }
    a.slots[i] = slot;
  }
  if (blockIdx.x == 0)
    for (int e = tid; e <= a.E; e += kThreads) a.offsets[e] = start[e];
  // rows without a choice: a segment's end, and what is behind the last one
  if (a.align > 1)
    for (int e = blockIdx.x * kWarps + wid; e < a.E; e += gridDim.x * kWarps)
      for (int32_t r = start[e] + total[e] + lane; r < start[e + 1]; r += 32) a.source[r] = -1;
  for (int64_t r = start[a.E] + (int64_t)blockIdx.x * kThreads + tid; r < a.capacity; r += (int64_t)gridDim.x * kThreads)
    a.source[r] = -1;
}

// ---- rows -----------------------------------------------------------------------

// A unit of a row, and as a register holds it.  (16-bit units in 32-bit registers: with
// uint16_t combine of 16384 x 1001 bf16, k 8, took 227 us and not 68.)
template <int BYTES> struct Unit;
template <> struct Unit<16> { using T = uint4; using Reg = uint4; };
template <> struct Unit<4> { using T = uint32_t; using Reg = uint32_t; };
template <> struct Unit<2> { using T = uint16_t; using Reg = uint32_t; };

// The elements of a unit.
template <int DT, int BYTES>
struct Packed {
  using E = Elem<DT>;
  using U = typename Unit<BYTES>::T;
  using Reg = typename Unit<BYTES>::Reg;
  static constexpr int N = BYTES / (int)sizeof(typename E::T);
  static __device__ __forceinline__ void unpack(const Reg u, float (&f)[N]) {
    if constexpr (BYTES == 16) E::unpack(u, f);
    else if constexpr (DT == SCAPE_F32) f[0] = __uint_as_float(u);
    else if constexpr (BYTES == 2) {
      const uint16_t h = (uint16_t)u;
      f[0] = E::load(&h);
    } else {
      const uint16_t lo = (uint16_t)u, hi = (uint16_t)(u >> 16);
      f[0] = E::load(&lo);
      f[1] = E::load(&hi);
    }
  }
  static __device__ __forceinline__ U pack(const float (&f)[N]) {
    if constexpr (BYTES == 16) return E::pack(f);
    else if constexpr (DT == SCAPE_F32) return __float_as_uint(f[0]);
    else if constexpr (BYTES == 2) return E::make(f[0]);
    else return E::pack2(f[0], f[1]);
  }
};

template <int BYTES>
__device__ __forceinline__ typename Unit<BYTES>::Reg zero_unit() {
  if constexpr (BYTES == 16) return make_uint4(0, 0, 0, 0);
  else return 0;
}
// Unit u of a row, 0 where there is none.
template <int BYTES>
__device__ __forceinline__ typename Unit<BYTES>::Reg unit_at(const typename Unit<BYTES>::T* row, int64_t u, bool there) {
  if constexpr (BYTES == 2) {
    uint32_t r = 0;
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n @p ld.global.u16 %0, [%1];\n}"
                 : "+r"(r)
                 : "l"(row + u), "r"((uint32_t)there)
                 : "memory");
    return r;
  } else {
    return there ? row[u] : zero_unit<BYTES>();
  }
}

struct RowArgs {
  const char* x;  // dispatch: tokens; combine, backward: rows by expert
  char* out;      // dispatch, backward: rows by expert; combine: tokens
  const char* d_out;
  int64_t stride;   // of a token's row, in bytes (dispatch)
  int64_t bytes;    // of a row
  int64_t tokens, rows;
  int k;
  int slices;       // parts of a row that are worked on apart (dispatch, combine)
  const int32_t* slots;
  const int32_t* source;
  const float* weights;
  float* d_weights;
  int64_t row_warps;  // dispatch, backward: warps for the tokens; the others look for empty rows
};

constexpr int kEmptyRows = 4;  // rows that such a warp looks at

template <int BYTES>
__device__ void clear_empty_rows(const RowArgs& a, int64_t item, int lane) {
  using U = typename Unit<BYTES>::T;
  const int64_t units = a.bytes / BYTES;
  for (int64_t r = item * kEmptyRows; r < min(a.rows, (item + 1) * kEmptyRows); r++) {
    if (a.source[r] >= 0) continue;
    U* out = reinterpret_cast<U*>(a.out + r * a.bytes);
    for (int64_t u = lane; u < units; u += 32) out[u] = (U)zero_unit<BYTES>();
  }
}

// A warp takes R units a lane of a token's row, and stores them k times.  Bound by HBM: 16384 x
// 2048 bf16 to 8 experts in 93 us (6.5 TB/s), stores for the most part.
template <int BYTES, int R>
__global__ __launch_bounds__(kThreads) void dispatch_rows(const RowArgs a) {
  using U = typename Unit<BYTES>::T;
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= a.row_warps) {
    clear_empty_rows<BYTES>(a, item - a.row_warps, lane);
    return;
  }
  const int64_t t = item / a.slices, u0 = (item % a.slices) * (32 * R) + lane, units = a.bytes / BYTES;
  int slot = lane < a.k ? a.slots[t * a.k + lane] : -1;
  if (slot >= a.rows) slot = -1;
  if (!__any_sync(kFull, slot >= 0)) return;  // (a token of no expert is not read)
  const U* x = reinterpret_cast<const U*>(a.x + t * a.stride);
  typename Unit<BYTES>::Reg v[R];
#pragma unroll
  for (int i = 0; i < R; i++) v[i] = unit_at<BYTES>(x, u0 + i * 32, u0 + i * 32 < units);
  for (int j = 0; j < a.k; j++) {
    const int s = __shfl_sync(kFull, slot, j);
    if (s < 0) continue;
    U* out = reinterpret_cast<U*>(a.out + s * a.bytes);
#pragma unroll
    for (int i = 0; i < R; i++)
      if (u0 + i * 32 < units) out[u0 + i * 32] = (U)v[i];
  }
}

// out[t] = sum over j of w_tj y[slot_tj], in this order, rounded once.  The loads of
// AHEAD choices are under way together: with those of one alone (64 bytes a lane) 605 MB
// took 138 us, with 128 bytes of four 90 (6.7 TB/s).
template <int DT, int BYTES, int R, int AHEAD>
__global__ __launch_bounds__(kThreads, 4) void combine_rows(const RowArgs a) {
  using P = Packed<DT, BYTES>;
  using U = typename P::U;
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= a.row_warps) return;
  const int64_t t = item / a.slices, u0 = (item % a.slices) * (32 * R) + lane, units = a.bytes / BYTES;
  int slot = -1;
  float w = 0.0f;
  if (lane < a.k) {
    slot = a.slots[t * a.k + lane];
    if (slot >= a.rows) slot = -1;
    if (slot >= 0) w = a.weights ? a.weights[t * a.k + lane] : 1.0f;
  }
  float acc[R][P::N];
#pragma unroll
  for (int i = 0; i < R; i++)
#pragma unroll
    for (int e = 0; e < P::N; e++) acc[i][e] = 0.0f;
  for (int j0 = 0; j0 < a.k; j0 += AHEAD) {
    typename P::Reg v[AHEAD][R];
#pragma unroll
    for (int j = 0; j < AHEAD; j++) {
      const int s = __shfl_sync(kFull, slot, (j0 + j) & 31);
      const bool on = s >= 0 && j0 + j < a.k;
      const U* y = reinterpret_cast<const U*>(a.x + (on ? s : 0) * a.bytes);
#pragma unroll
      for (int i = 0; i < R; i++) v[j][i] = unit_at<BYTES>(y, u0 + i * 32, on && u0 + i * 32 < units);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; j++) {
      const float wj = __shfl_sync(kFull, w, (j0 + j) & 31);  // (no choice: 0 times 0)
#pragma unroll
      for (int i = 0; i < R; i++) {
        float f[P::N];
        P::unpack(v[j][i], f);
#pragma unroll
        for (int e = 0; e < P::N; e++) acc[i][e] = __fmaf_rn(wj, f[e], acc[i][e]);
      }
    }
  }
  U* out = reinterpret_cast<U*>(a.out + t * a.bytes);
#pragma unroll
  for (int i = 0; i < R; i++)
    if (u0 + i * 32 < units) out[u0 + i * 32] = P::pack(acc[i]);
}

// dy[slot] = w dout[t], dw = <dout[t], y[slot]>.  A warp has two choices of a token, whose
// row it loads once for both; the warps of the token's other choices find it in L1.
// (With one choice a warp, and half of the loads under way: 128 us for 696 MB; so, 114.)
constexpr int kPair = 2;
template <int DT, int BYTES, int R>
__global__ __launch_bounds__(kThreads, 4) void combine_grad(const RowArgs a) {
  using P = Packed<DT, BYTES>;
  using U = typename P::U;
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= a.row_warps) {
    clear_empty_rows<BYTES>(a, item - a.row_warps, lane);
    return;
  }
  const int pairs = (a.k + kPair - 1) / kPair;
  const int64_t t = item / pairs, units = a.bytes / BYTES;
  const int j0 = (int)(item - t * pairs) * kPair;
  bool on[kPair];
  float w[kPair], dot[kPair];
  const U* y[kPair];
  U* dy[kPair];
#pragma unroll
  for (int c = 0; c < kPair; c++) {
    const int s = j0 + c < a.k ? a.slots[t * a.k + j0 + c] : -1;
    on[c] = s >= 0 && s < a.rows;
    w[c] = on[c] ? a.weights[t * a.k + j0 + c] : 0.0f;
    y[c] = reinterpret_cast<const U*>(a.x + (on[c] ? s : 0) * a.bytes);
    dy[c] = reinterpret_cast<U*>(a.out + (on[c] ? s : 0) * a.bytes);
    dot[c] = 0.0f;
  }
  bool any = false;
#pragma unroll
  for (int c = 0; c < kPair; c++) any |= on[c];
  if (any) {  // (a token without a choice is not read)
    const U* g = reinterpret_cast<const U*>(a.d_out + t * a.bytes);
    for (int64_t u0 = lane; u0 < units; u0 += 32 * R) {
      typename P::Reg vy[kPair][R], vg[R];
#pragma unroll
      for (int i = 0; i < R; i++) {
        const bool in = u0 + i * 32 < units;
        vg[i] = unit_at<BYTES>(g, u0 + i * 32, in);
#pragma unroll
        for (int c = 0; c < kPair; c++) vy[c][i] = unit_at<BYTES>(y[c], u0 + i * 32, in && on[c]);
      }
#pragma unroll
      for (int i = 0; i < R; i++) {
        float fg[P::N];
        P::unpack(vg[i], fg);
#pragma unroll
        for (int c = 0; c < kPair; c++) {
          float fy[P::N], d[P::N];
          P::unpack(vy[c][i], fy);
#pragma unroll
          for (int e = 0; e < P::N; e++) {
            dot[c] = __fmaf_rn(fg[e], fy[e], dot[c]);
            d[e] = fg[e] * w[c];
          }
          if (on[c] && u0 + i * 32 < units) dy[c][u0 + i * 32] = P::pack(d);
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kPair; c++) {
    float d = dot[c];
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(kFull, d, o);
    if (lane == 0 && a.d_weights && j0 + c < a.k) a.d_weights[t * a.k + j0 + c] = on[c] ? d : 0.0f;
  }
}

int check_plan(uint64_t tokens, int k, int experts, int align, uint64_t& capacity, uint64_t& bytes) {
  if (experts < 1 || experts > kMaxExperts)
    return fail(SCAPE_EINVAL, "experts=%d must be in [1, %d]", experts, kMaxExperts);
  if (k < 1 || k > kMaxChoices) return fail(SCAPE_EINVAL, "k=%d outside [1, %d]", k, kMaxChoices);
  if (align < 1 || align > 65536) return fail(SCAPE_EINVAL, "align=%d must be in [1, 65536]", align);
  if (tokens >= (1ull << 31)) return fail(SCAPE_EINVAL, "tokens must be < 2^31");
  const uint64_t n = tokens * (uint64_t)k;
  capacity = n + std::min<uint64_t>((uint64_t)experts, n) * (uint64_t)(align - 1);
  if (capacity >= (1ull << 31)) return fail(SCAPE_EINVAL, "the plan must have < 2^31 rows");
  const uint64_t chunks = (n + kChunk - 1) / kChunk;
  bytes = chunks > 1 ? (chunks + 1) * (uint64_t)experts * 4 : 0;
  return SCAPE_OK;
}

// The widest unit that a row's length and all addresses are multiples of.
int unit_of(int dtype, uint64_t bytes, std::initializer_list<uintptr_t> at) {
  uintptr_t all = bytes;
  for (uintptr_t p : at) all |= p;
  return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : (int)size_of(dtype);
}

// Units of a row that a lane has in flight, of 16 bytes and of fewer: dispatch; combine,
// of each choice; its backward pass, of each choice and the token's row.
constexpr int kUnits16 = 4, kUnitsSmall = 8, kBack16 = 3, kBack4 = 4, kBack2 = 8;
// (two choices leave room for more of each)
int combine_units(int unit, int k) { return unit == 16 ? (k <= 2 ? 4 : 2) : unit == 4 ? 4 : 8; }

// As many 16-byte units a lane, up to "most", as divide a row of "bytes" into equal rounds
// (1280 bf16 elements: 3 and 2 of them, not 4 and 1).
int units16_of(uint64_t bytes, int most) {
  const int all = (int)((bytes / 16 + 31) / 32), rounds = (all + most - 1) / most;
  return (all + rounds - 1) / rounds;
}

int check_rows(int dtype, uint64_t tokens, int k, uint64_t rows, uint64_t dim) {
  if (dtype < SCAPE_BF16 || dtype > SCAPE_F32) return fail(SCAPE_EINVAL, "unknown dtype %d", dtype);
  if (k < 1 || k > kMaxChoices) return fail(SCAPE_EINVAL, "k=%d outside [1, %d]", k, kMaxChoices);
  if (tokens >= (1ull << 31) || rows >= (1ull << 31) || tokens * (uint64_t)k >= (1ull << 31))
    return fail(SCAPE_EINVAL, "tokens x k and rows must be < 2^31");
  if (dim < 1 || dim >= (1ull << 24)) return fail(SCAPE_EINVAL, "dim=%llu must be in [1, 2^24)", (unsigned long long)dim);
  return SCAPE_OK;
}

void fill(RowArgs& a, int dtype, uint64_t tokens, int k, uint64_t rows, uint64_t dim) {
  a.bytes = (int64_t)(dim * size_of(dtype));
  a.tokens = (int64_t)tokens;
  a.rows = (int64_t)rows;
  a.k = k;
}

// Parts of a row of "bytes", "units" units a lane each.
int slices_of(int64_t bytes, int unit, int units) {
  const int64_t part = 32 * (int64_t)unit * units;
  return (int)((bytes + part - 1) / part);
}

bool grid_of(int64_t warps, unsigned& grid) {
  const int64_t g = (warps + kWarps - 1) / kWarps;
  grid = (unsigned)g;
  return g < (1ll << 31);
}

}  // namespace
}  // namespace scape

SCAPE_API int scape_expert_plan_sizes(uint64_t tokens, int k, int experts, int align, uint64_t* capacity,
                                      uint64_t* workspace_bytes) {
  using namespace scape;
  if (!capacity || !workspace_bytes) return fail(SCAPE_EINVAL, "capacity and workspace_bytes are required");
  *capacity = *workspace_bytes = 0;
  uint64_t c, b;
  if (int rc = check_plan(tokens, k, experts, align, c, b)) return rc;
  *capacity = c;
  *workspace_bytes = b;
  return SCAPE_OK;
}

SCAPE_API int scape_expert_plan(const int32_t* idx, uint64_t tokens, int k, int experts, int align,
                                int32_t* offsets, int32_t* slots, int32_t* source, uint32_t* bad_count,
                                void* workspace, uint64_t workspace_bytes, void* stream) {
  using namespace scape;
  uint64_t capacity, need;
  if (int rc = check_plan(tokens, k, experts, align, capacity, need)) return rc;
  if (!offsets || (tokens > 0 && (!idx || !slots || !source)))
    return fail(SCAPE_EINVAL, "idx, offsets, slots and source are required");
  if (misaligned(idx, 4) || misaligned(offsets, 4) || misaligned(slots, 4) || misaligned(source, 4) ||
      misaligned(bad_count, 4))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  if (need && (!workspace || misaligned(workspace, 16) || workspace_bytes < need))
    return fail(SCAPE_EINVAL, "workspace must be %llu bytes, 16-byte aligned", (unsigned long long)need);
  PlanArgs a{};
  a.idx = idx;
  a.n = (int64_t)(tokens * (uint64_t)k);
  a.E = experts;
  a.align = align;
  a.chunks = (a.n + kChunk - 1) / kChunk;
  a.capacity = (int64_t)capacity;
  a.offsets = offsets;
  a.slots = slots;
  a.source = source;
  a.bad = bad_count;
  a.totals = static_cast<int32_t*>(workspace);
  a.counts = a.totals + experts;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.chunks <= 1) {
    e = launch_behind(place_choices<true>, 1, kThreads, s, a);
  } else {
    e = launch_behind(place_counts, (unsigned)a.chunks, kThreads, s, a);
    if (e != cudaSuccess) return fail(SCAPE_ECUDA, "place_counts: %s", cudaGetErrorString(e));
    e = launch_behind(place_scan, (unsigned)((experts + 31) / 32), 1024, s, a);
    if (e != cudaSuccess) return fail(SCAPE_ECUDA, "place_scan: %s", cudaGetErrorString(e));
    e = launch_behind(place_choices<false>, (unsigned)a.chunks, kThreads, s, a);
  }
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "place_choices: %s", cudaGetErrorString(e));
}

SCAPE_API int scape_expert_dispatch(const void* x, int dtype, uint64_t tokens, uint64_t dim,
                                    uint64_t row_stride, int k, const int32_t* slots,
                                    const int32_t* source, uint64_t rows, void* out, void* stream) {
  using namespace scape;
  if (int rc = check_rows(dtype, tokens, k, rows, dim)) return rc;
  if (row_stride < dim || row_stride >= (1ull << 32)) return fail(SCAPE_EINVAL, "row_stride must be >= dim and < 2^32");
  if (rows == 0) return SCAPE_OK;
  if ((tokens > 0 && (!x || !slots)) || !source || !out)
    return fail(SCAPE_EINVAL, "x, slots, source and out are required");
  const uint64_t es = size_of(dtype);
  if (misaligned(x, es) || misaligned(out, es) || misaligned(slots, 4) || misaligned(source, 4))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  if (tokens && ranges_meet(x, ((tokens - 1) * row_stride + dim) * es, out, rows * dim * es))
    return fail(SCAPE_EINVAL, "out must not overlap x");
  RowArgs a{};
  const int unit = unit_of(dtype, dim * es, {row_stride * es, reinterpret_cast<uintptr_t>(x), reinterpret_cast<uintptr_t>(out)});
  const int units = unit == 16 ? units16_of(dim * es, kUnits16) : kUnitsSmall;
  fill(a, dtype, tokens, k, rows, dim);
  a.slices = slices_of(a.bytes, unit, units);
  a.x = static_cast<const char*>(x);
  a.out = static_cast<char*>(out);
  a.stride = (int64_t)(row_stride * es);
  a.slots = slots;
  a.source = source;
  a.row_warps = a.tokens * a.slices;
  unsigned grid;
  if (!grid_of(a.row_warps + (a.rows + kEmptyRows - 1) / kEmptyRows, grid)) return fail(SCAPE_EINVAL, "too many rows");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (unit == 16)
    e = units == 1   ? launch_behind(dispatch_rows<16, 1>, grid, kThreads, s, a)
        : units == 2 ? launch_behind(dispatch_rows<16, 2>, grid, kThreads, s, a)
        : units == 3 ? launch_behind(dispatch_rows<16, 3>, grid, kThreads, s, a)
                     : launch_behind(dispatch_rows<16, kUnits16>, grid, kThreads, s, a);
  else if (unit == 4) e = launch_behind(dispatch_rows<4, kUnitsSmall>, grid, kThreads, s, a);
  else e = launch_behind(dispatch_rows<2, kUnitsSmall>, grid, kThreads, s, a);
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "dispatch_rows: %s", cudaGetErrorString(e));
}

namespace scape {
namespace {
template <int DT>
cudaError_t launch_combine(const RowArgs& a, int unit, unsigned grid, bool back, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (unit == 16) {
    const int units = units16_of((uint64_t)a.bytes, kBack16);
    if (back)
      e = units == 1   ? launch_behind(combine_grad<DT, 16, 1>, grid, kThreads, s, a)
          : units == 2 ? launch_behind(combine_grad<DT, 16, 2>, grid, kThreads, s, a)
                       : launch_behind(combine_grad<DT, 16, kBack16>, grid, kThreads, s, a);
    else
      e = a.k <= 2 ? launch_behind(combine_rows<DT, 16, 4, 2>, grid, kThreads, s, a)
                   : launch_behind(combine_rows<DT, 16, 2, 4>, grid, kThreads, s, a);
  } else if (unit == 4) {
    if (back) e = launch_behind(combine_grad<DT, 4, kBack4>, grid, kThreads, s, a);
    else e = launch_behind(combine_rows<DT, 4, 4, 4>, grid, kThreads, s, a);
  } else if constexpr (DT != SCAPE_F32) {
    if (back) e = launch_behind(combine_grad<DT, 2, kBack2>, grid, kThreads, s, a);
    else e = launch_behind(combine_rows<DT, 2, 8, 4>, grid, kThreads, s, a);
  }
  return e;
}
cudaError_t launch_combine_any(int dtype, const RowArgs& a, int unit, unsigned grid, bool back, cudaStream_t s) {
  if (dtype == SCAPE_BF16) return launch_combine<SCAPE_BF16>(a, unit, grid, back, s);
  if (dtype == SCAPE_F16) return launch_combine<SCAPE_F16>(a, unit, grid, back, s);
  return launch_combine<SCAPE_F32>(a, unit, grid, back, s);
}
}  // namespace
}  // namespace scape

SCAPE_API int scape_expert_combine(const void* y, int dtype, uint64_t rows, uint64_t dim,
                                   const int32_t* slots, const float* weights, uint64_t tokens, int k,
                                   void* out, void* stream) {
  using namespace scape;
  if (int rc = check_rows(dtype, tokens, k, rows, dim)) return rc;
  if (tokens == 0) return SCAPE_OK;
  if ((rows > 0 && !y) || !slots || !out) return fail(SCAPE_EINVAL, "y, slots and out are required");
  const uint64_t es = size_of(dtype);
  if (misaligned(y, es) || misaligned(out, es) || misaligned(slots, 4) || misaligned(weights, 4))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  if (ranges_meet(y, rows * dim * es, out, tokens * dim * es)) return fail(SCAPE_EINVAL, "out must not overlap y");
  RowArgs a{};
  const int unit = unit_of(dtype, dim * es, {reinterpret_cast<uintptr_t>(y), reinterpret_cast<uintptr_t>(out)});
  fill(a, dtype, tokens, k, rows, dim);
  a.slices = slices_of(a.bytes, unit, combine_units(unit, k));
  a.x = static_cast<const char*>(y);
  a.out = static_cast<char*>(out);
  a.slots = slots;
  a.weights = weights;
  a.row_warps = a.tokens * a.slices;
  unsigned grid;
  if (!grid_of(a.row_warps, grid)) return fail(SCAPE_EINVAL, "too many rows");
  const cudaError_t e = launch_combine_any(dtype, a, unit, grid, false, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "combine_rows: %s", cudaGetErrorString(e));
}

SCAPE_API int scape_expert_combine_backward(const void* d_out, const void* y, int dtype, uint64_t rows,
                                            uint64_t dim, const int32_t* slots, const int32_t* source,
                                            const float* weights, uint64_t tokens, int k, void* d_y,
                                            float* d_weights, void* stream) {
  using namespace scape;
  if (int rc = check_rows(dtype, tokens, k, rows, dim)) return rc;
  if (rows == 0 && tokens == 0) return SCAPE_OK;
  if ((tokens > 0 && (!d_out || !slots || !weights)) || (rows > 0 && (!y || !source || !d_y)))
    return fail(SCAPE_EINVAL, "d_out, y, slots, source, weights and d_y are required");
  const uint64_t es = size_of(dtype);
  if (misaligned(d_out, es) || misaligned(y, es) || misaligned(d_y, es) || misaligned(slots, 4) ||
      misaligned(source, 4) || misaligned(weights, 4) || misaligned(d_weights, 4))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  if (ranges_meet(d_y, rows * dim * es, d_out, tokens * dim * es) || ranges_meet(d_y, rows * dim * es, y, rows * dim * es))
    return fail(SCAPE_EINVAL, "d_y must not overlap d_out or y");
  RowArgs a{};
  const int unit = unit_of(dtype, dim * es, {reinterpret_cast<uintptr_t>(y), reinterpret_cast<uintptr_t>(d_out),
                                             reinterpret_cast<uintptr_t>(d_y)});
  fill(a, dtype, tokens, k, rows, dim);
  a.x = static_cast<const char*>(y);
  a.d_out = static_cast<const char*>(d_out);
  a.out = static_cast<char*>(d_y);
  a.slots = slots;
  a.source = source;
  a.weights = weights;
  a.d_weights = d_weights;
  a.row_warps = a.tokens * ((a.k + kPair - 1) / kPair);
  unsigned grid;
  if (!grid_of(a.row_warps + (a.rows + kEmptyRows - 1) / kEmptyRows, grid)) return fail(SCAPE_EINVAL, "too many rows");
  const cudaError_t e = launch_combine_any(dtype, a, unit, grid, true, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SCAPE_OK : fail(SCAPE_ECUDA, "combine_grad: %s", cudaGetErrorString(e));
}
