// Softmax cross entropy of hidden states through an output matrix, without the
// logits in memory (scape_linear_ce).
//
//   l_tv = h_t . W_v;  loss_t = w_t (log sum_v exp l_tv - l_{t, y_t})
//   G_tv = w_t (exp(l_tv - lse_t) - [v = y_t]);  dH = G W;  dW = G^T H
//
// Four products on the tensor cores (16-bit operands, fp32 accumulators in tensor
// memory), one kernel for all:
//   LOSS  H W^T: the maximum and the sum of exponentials of every row of a tile, and
//         the label's logit; for a gradient also the logits themselves, as distances
//         from that maximum, for as many words as there is room for
//   GRAD  the same product again, for a piece of the vocabulary without such room: G of
//         that piece
//   BACK  G W, added up over the pieces in fp32, and G^T H, complete for the piece's
//         words: the tiles of both in one launch
// With GRAD a gradient costs 8 T D V operations, without it 6.  What LOSS keeps of a
// logit is its distance from the maximum of its 128 words, in 16 bits (Kept), and G
// takes its place (grad_kept).
//
// Rows without a term (no label, weight 0) are left out: the others are copied
// together first, so that neither time nor the gradients depend on what they hold.
//
// G is rounded to the operands' type: its entries carry half a step of it, as the
// results do.  Row weights are first divided by the largest of them, and the results
// multiplied by it: where all weights are the same, as those of a mean, the labels'
// entries, w (p - 1), are then next to -1 and not all rounded the same way (of bf16
// results 4.5e-3 instead of 1.8e-3 off).  For fp16 they are multiplied by 2^14, too,
// which keeps small entries clear of the end of its range.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>

#include "host.cuh"
#include "objective.cuh"
#include "scape_kernels.cuh"
#include "tc.cuh"

#define SCAPE_API extern "C" __attribute__((visibility("default")))

namespace scape {
namespace {

using namespace tc;

enum Job { LOSS, GRAD, BACK };

constexpr int kM = 128, kN = 256, kK = 64;  // a CTA's tile; 64 elements are one swizzled row
// A pair of CTAs has a tile of 256 x 256: each copies its own 128 rows of A and half of
// the columns of B, a third less than alone.  The tiles of K on their way fill the same
// memory either way; where rows or words are few, more of them.
template <int CG>
struct Shape {
  static constexpr int kRows = kM * CG, kCols = kN / CG;  // rows of a tile; columns of B that a CTA copies
  static constexpr int kMaxStages = CG == 2 ? 6 : 16;
};
constexpr uint32_t kRing = 196608;  // all stages: 6 of a pair's (32 KB), 4 of a CTA's alone (48 KB)
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;  // copies, products, allocation, one idle; epilogue
constexpr uint32_t kOutBytes = 4096;            // a warp's results on their way out: 32 rows of 128 bytes
constexpr uint32_t kSmem = kRing + kEpiWarps * kOutBytes + 1024;
constexpr int kGroup = 16;                      // tiles of rows that walk along the other dimension together
constexpr uint64_t kTileFloats = (uint64_t)kM * kN;

struct CeArgs {
  // rows with a term, together
  const int32_t* map;      // their places among the caller's
  const int32_t* label;
  const float* weight;
  float* label_logit;
  float* left;             // what rounding took from the label's entry of G
  const void* w;           // vocab x D
  int64_t w_stride;
  float2* parts;           // cap x n_parts (two for a tile of words): maximum, sum of exponentials
  int n_parts;
  float2* stats;           // cap: maximum, log2 of the sum
  int32_t* live;
  float* scale;            // of the weights, and its reciprocal
  uint32_t* status;        // 0, or a wait ran out
  float* loss;             // caller's
  int64_t rows, cap;       // caller's rows; rounded up (Cut)
  int D, V;
  int bn;                  // words of a tile (LOSS, GRAD)
  int bm;                  // rows of a CTA's tile of H or G that are copied
  int keep;                // words below this are kept (LOSS)
  // the piece of the vocabulary
  int v0, vn;
  int piece;               // words of a piece, all but the last one
  int64_t g0;              // its first row in the buffer of G
  void* g;
  // sums of tiles in fp32, a float4 of a row's columns 4 j to 4 j + 3 at [j][row]
  float* acc;              // dH, over the pieces: all tiles
  float* tail;             // the parts of split tiles, of dH and behind them of dW
  int grid;                // CTAs, or pairs of them, of BACK
  int first, last;
  int early;               // LOSS: no more than one row of tiles
#ifdef SCAPE_DEBUG_CHECKS
  int lost;                // test hook: in this job (1 + Job) the first products wait for what nobody sends
#endif
  void* d_hidden;
  int64_t dh_stride;
  void* d_weight;
  int64_t dw_stride;
};

__device__ __forceinline__ int up_div(int x, int y) { return (x + y - 1) / y; }

// Tiles of a product, in the order in which they are worked on: up to kGroup rows of tiles
// at a time, down first, in groups of equal height.  (17 rows of tiles, loss of 4352 x 32000, dim
// 2048: 322 us, with groups of 16 and of one 329 to 335.)
struct Tiles {
  int mt, nt, kb;  // kb: blocks of the sum
  __device__ __forceinline__ int count() const { return mt * nt; }
  __device__ __forceinline__ void place(int tile, int& m, int& n) const {
    const int groups = up_div(mt, kGroup), high = up_div(mt, groups);
    const int g = tile / (high * nt), in = tile - g * high * nt;
    const int rows = min(high, mt - g * high);
    n = in / rows;
    m = g * high + in - n * rows;
  }
};

// A unit of work: a tile, or a part of its sum.
struct Unit {
  int m, n, k0, k1;
  int tile;
  int part;  // its place among the parts of its product, -1 for a whole tile
  bool dw;   // BACK: of dW
};

// The tensor cores cut off what an addition to an accumulator loses, always towards 0, so the
// sums over the vocabulary and over the rows are taken in chains of at most so many blocks
// (8192 terms, 512 additions), added up in fp32 by the epilogue, which has the time.  In one
// chain the fp16 d_hidden of 32000 words with a common direction was 2.99e-4 off and is
// 2.30e-4 (2.08e-4: its own rounding), d_weight of 8 M rows 3.1e-3 and is 2.0e-4.
constexpr int kChain = 128;
// Sums over dim, of logits, are taken in chains where they are long (LONG: dim > kLongDim): of 1024
// terms, 64 additions, added up in the registers of the epilogue, which for that has those
// of the other warps.  Losses of 1000 rows, 32000 words, dim 4096: 1.6e-6 (bf16) and 1.9e-6 (fp16) off in one
// chain, 3.8e-7 and 4.6e-7 so (fp32 throughout: 4.3e-7 and 5.1e-7); dim 1280 in one 3.7e-7
// and 5.0e-7.  It costs 4 % of the cycles of a loss of dim 2048 whose logits are kept, else nothing
// (the epilogue's instructions count: chains added up by 512 of them a warp's tile instead of 64 cost 3 %
// and 10 %; so do spills in the thread that issues the products, with 72 registers for it and 216).
constexpr int kLossChain = 16, kLongDim = 1280;
constexpr int kRegsOthers = 88, kRegsEpilogue = 208;  // of a thread: 128 x 88 + 256 x 208 = 384 x 168 at the launch
template <int JOB, bool LONG>
__device__ __forceinline__ int chain_end(const Unit& u, int k) {  // ... of the chain that begins at k
  return JOB == BACK ? min(u.k1, k + kChain) : LONG ? min(u.k1, k + kLossChain) : u.k1;
}

// The units of a CTA (or pair), one after the other.
template <int JOB, int CG>
struct Work {
  Tiles t;
  __device__ __forceinline__ Work(const CeArgs& a, int live)
      : t{up_div(live, Shape<CG>::kRows), up_div(a.vn, a.bn), up_div(a.D, kK)} {}
  __device__ __forceinline__ bool get(int me, int all, int j, Unit& u) const {
    u.tile = me + j * all;
    if (u.tile >= t.count()) return false;
    t.place(u.tile, u.m, u.n);
    u.k0 = 0;
    u.k1 = t.kb;
    u.part = -1;
    u.dw = false;
    return true;
  }
};

// BACK: first the tiles of dH, whose sums are long, then those of dW.  Where the tiles of
// dH do not go evenly into the CTAs, those that have one less begin with as many tiles of
// dW as that one takes.  So the CTAs end together, which two launches do not let them:
// with 55 tiles of dH for 76 pairs of CTAs and 625 of dW (2723 rows, 32000 x 1280) a whole
// gradient took 555 us in two and takes 530 in one.  Split, and added up by join_parts, are
// the tiles of dH where they are too few and too long for that, and those of dW that
// would be a last round by themselves.
constexpr int kMaxParts = 2;         // of each product, per CTA
// (Where rows make several chains of a tile of dW, the second half of the places for parts of dH
// holds the CTAs' sums of chains; where dH is not split, it is free anyway.)
// What a unit costs beside its blocks, in blocks: of pairs, of CTAs alone, whose blocks wait
// for HBM; and what writing and adding up a CTA's part costs, on all CTAs.  Gradients with 32000 words in
// a graph, us, with 4 and 1.5 | 1 and 0.5 | 8 and 4:
//   16 rows    dim 1024  73.8 |  78.1 |  73.8   dim 4096 177.6 | 187.6 | 184.3
//   200 rows   dim 1024  96.3 | 102.7 | 102.5   dim 4096 222.0 | 244.4 | 233.7
//   512 rows   dim 2048 179.5 | 191.6 | 189.5   dim 4096 312.9 | 328.7 | 332.3
// (100 rows of dim 4096: 195, 191, 205; from 1300 rows on all three within noise)
constexpr float kUnitCost = 4.0f, kUnitCostOne = 1.5f, kPartCost = 0.14f;
template <int CG>
struct Work<BACK, CG> {
  Tiles h, w;
  int split_h;          // parts of every tile of dH
  int each, more;       // units of dH of every CTA; CTAs with one more
  int early;            // tiles of dW that the others begin with
  int whole, split_w;   // tiles of dW that are not split; parts of the others
  __device__ __forceinline__ Work(const CeArgs& a, int live) {
    constexpr int kRows = Shape<CG>::kRows;
    const int all = a.grid;
    h = {up_div(live, kRows), up_div(a.D, kN), up_div(a.vn, kK)};
    w = {up_div(a.vn, kRows), up_div(a.D, kN), up_div(live, kK)};
    constexpr float kUnit = CG == 2 ? kUnitCost : kUnitCostOne;
    const float cost_w = (float)w.kb + kUnit;
    split_h = 1;
    float best = 0.0f;
    const int most = w.kb > kChain ? all : kMaxParts * all;
    for (int s = 1; s <= 32 && (s == 1 || (s * h.count() <= most && 8 * s <= h.kb)); s++) {
      const int n = s * h.count();
      const float unit = (float)h.kb / (float)s + kUnit;
      const float even = ((float)n * unit + (float)w.count() * cost_w) / (float)all;
      const float last = (float)up_div(n, all) * unit;
      const float cost = fmaxf(even, last) + (s > 1 ? kPartCost * (float)(n * CG) : 0.0f);
      if (s == 1 || cost < best) {
        best = cost;
        split_h = s;
      }
      if (h.count() >= all) break;
    }
    const int n = split_h * h.count();
    each = n / all;
    more = n - each * all;
    const float unit = (float)h.kb / (float)split_h + kUnit;
    early = more ? min((int)(unit / cost_w + 0.5f), w.count() / (all - more)) : 0;
    const int left = w.count() - early * (all - more), rest = left % all;
    whole = w.count();
    split_w = 1;
    float round = 0.9f;  // the last one, of a whole one
    for (int s = 2; s <= 16 && rest && s * rest <= kMaxParts * all && 8 * s <= w.kb; s++) {
      const float cost = (float)up_div(s * rest, all) / (float)s + kPartCost * (float)(s * rest * CG) / cost_w;
      if (cost < round) {
        round = cost;
        split_w = s;
      }
    }
    if (split_w > 1) whole -= rest;
  }
  __device__ __forceinline__ int rest() const { return w.count() - whole; }
  __device__ __forceinline__ bool get(int me, int all, int j, Unit& u) const {
    const bool has_more = me < more;
    const int own = each + has_more;
    u.dw = j >= own;
    if (!u.dw) {
      const int i = me + j * all, s = i / h.count();
      u.tile = i - s * h.count();
      h.place(u.tile, u.m, u.n);
      u.k0 = (int)((int64_t)h.kb * s / split_h);
      u.k1 = (int)((int64_t)h.kb * (s + 1) / split_h);
      u.part = split_h > 1 ? i : -1;
      return true;
    }
    j -= own;
    const int others = all - more, first = early * others;
    int i;
    if (has_more) i = first + j * all + me;
    else if (j < early) i = j * others + me - more;
    else i = first + (j - early) * all + me;
    if (i < whole) {
      u.tile = i;
      u.k0 = 0;
      u.k1 = w.kb;
      u.part = -1;
    } else {
      if (i >= whole + rest() * split_w) return false;
      const int p = i - whole, s = p / rest();
      u.tile = whole + p - s * rest();
      u.k0 = (int)((int64_t)w.kb * s / split_w);
      u.k1 = (int)((int64_t)w.kb * (s + 1) / split_w);
      u.part = p;
    }
    w.place(u.tile, u.m, u.n);
    return true;
  }
  // Where a CTA adds up the chains of a whole tile.
  static __device__ __forceinline__ float* chains_at(const CeArgs& a, int me, int rank) {
    return part_at(a, false, a.grid + me, rank);
  }
  // Where the parts of a CTA's half of a unit are.
  static __device__ __forceinline__ float* part_at(const CeArgs& a, bool dw, int part, int rank) {
    return a.tail + ((int64_t)((dw ? kMaxParts * a.grid : 0) + part) * CG + rank) * (int64_t)kTileFloats;
  }
};

// A number as the operands' type holds it.
template <int DT>
__device__ __forceinline__ float rounded(float x) {
  const typename Elem<DT>::T t = Elem<DT>::make(x);
  return Elem<DT>::load(&t);
}

// Eight columns of a row of dH, from d on, with the part of the label's entry that its
// rounding in G took away.  That entry is the largest of most rows, next to -w, and
// without this its rounding would be most of the error of dH.
template <int DT>
__device__ __forceinline__ void add_left(const CeArgs& a, int r, int d, float (&f)[8]) {
  using E = Elem<DT>;
  const typename E::T* w = static_cast<const typename E::T*>(a.w) + (int64_t)a.label[r] * a.w_stride + d;
  float x[8];
  E::unpack(ld_row_u4(w), x);
  const float left = a.left[r];
#pragma unroll
  for (int j = 0; j < 8; j++) f[j] = __fmaf_rn(left, x[j], f[j]);
}

// Vector v of the lane's row in the warp's buffer, whose rows hold 64 results in eight
// swizzled vectors (as the copy engine expects them).
__device__ __forceinline__ uint32_t staged(uint32_t out, int lane, int v) {
  return out + lane * 128 + (uint32_t)((v ^ (lane & 7)) * 16);
}
// 32 results of a row into the buffer; "side" is the half.
template <int DT>
__device__ __forceinline__ void stage32(uint32_t out, int lane, int side, const float (&f)[32]) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; i++) g[i] = f[8 * j + i];
    put_smem(staged(out, lane, side * 4 + j), Elem<DT>::pack(g));
  }
}

// What is kept of a logit: its distance s <= 0 from the maximum of its 128 words, in units of
// ln 2, as a code of 16 bits that is linear in s, with finer steps from the knee up to 0 than
// from there down to where G holds no more of 2^s (code 0).  A step of s is that step times
// ln 2 of the exponential, wherever it is; half of one is
//   bf16  2^-11.5 down to s = -48, 2^-9.2 down to -128   (G: 2^-8)
//   fp16  2^-13.1 down to s = -12, 2^-11.5 down to -40   (G: 2^-11, of its own least step below -28)
// (Exponentials in fp16 lost their bits from s = -29 on and all of them from -40, and their
// rounding was as large as that of an fp16 G: the gradients of 2000 words that are no label,
// 300 rows, were 2.93e-4 off and are 2.63e-4.)
template <int DT> struct Kept;
template <> struct Kept<SCAPE_BF16> {  // codes of the two lines at s = 0, codes a unit
  static constexpr float kHigh = 1024.0f, kLow = 204.75f, kLow0 = 26211.0f;
};
template <> struct Kept<SCAPE_F16> {
  static constexpr float kHigh = 3064.0f, kLow = 1024.0f, kLow0 = 41055.0f;
};
constexpr float kHigh0 = 65535.0f;
constexpr float kInt = 8388608.0f;  // 2^23: a sum with it is rounded to a whole number, its low bits

// Two codes as the low 16 bits of two floats (the larger one of the two lines, at least 0).
template <int DT>
__device__ __forceinline__ uint32_t keep2(pair_t s) {
  using K = Kept<DT>;
  const pair_t hi = fma2(s, pair(K::kHigh, K::kHigh), pair(kInt + kHigh0, kInt + kHigh0));
  const pair_t lo = fma2(s, pair(K::kLow, K::kLow), pair(kInt + K::kLow0, kInt + K::kLow0));
  const float a = fmaxf(fmaxf(hi.x, lo.x), kInt), b = fmaxf(fmaxf(hi.y, lo.y), kInt);
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
}
// Eight exponentials 2^(s + by) times "scale" of a vector of codes.
template <int DT>
__device__ __forceinline__ void kept8(const uint4 v, float by, float scale, float (&f)[8]) {
  using K = Kept<DT>;
  const float hi0 = by - kHigh0 / K::kHigh, lo0 = by - K::kLow0 / K::kLow;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const pair_t c = add2(pair(__uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7610)),
                               __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7632))), pair(-kInt, -kInt));
    const pair_t hi = fma2(c, pair(1.0f / K::kHigh, 1.0f / K::kHigh), pair(hi0, hi0));
    const pair_t lo = fma2(c, pair(1.0f / K::kLow, 1.0f / K::kLow), pair(lo0, lo0));
    const pair_t e = mul2(ex2_2(pair(fminf(hi.x, lo.x), fminf(hi.y, lo.y))), pair(scale, scale));
    f[2 * i] = e.x;
    f[2 * i + 1] = e.y;
  }
}

// What a warp of the epilogue does with its 32 rows and 128 columns of a unit, in tensor
// memory at "tmem" ("empty": there were no products, all is 0).  BACK: begin, end: of the
// unit's chains this is the first, the last; me: the CTA (or pair).  LONG: the sums of all
// chains, in registers.
template <int JOB, int DT, int CG, bool KEEP, bool LONG>
__device__ __forceinline__ void epilogue(const CeArgs& a, const CUtensorMap* map_out, const Unit& u, int live, int me,
                                         int rank, int half, int quarter, int lane, uint32_t tmem, bool empty, bool begin,
                                         bool end, uint32_t out, float (&sums)[2][LONG ? 64 : 1]) {
  const int r0 = u.m * Shape<CG>::kRows + rank * kM + quarter * 32, r = r0 + lane;
  float f[32];
  auto fetch = [&](int c) {
    if (empty) {
#pragma unroll
      for (int i = 0; i < 32; i++) f[i] = 0.0f;
    } else {
      tmem_load(tmem + (uint32_t)(32 * c), f);
    }
  };
  // (both halves of a row are in the buffer: 64 columns go out from column x)
  auto send = [&](int x, int y) {
    store_fence();
    __syncwarp();
    if (lane == 0) store_box(map_out, x, y, out);
  };
  auto reuse = [&]() {
    if (lane == 0) store_read();
    __syncwarp();
  };
  if constexpr (JOB == LOSS) {
    const int label = r < live ? a.label[r] : -1;
    const int end = min(a.V, (u.n + 1) * a.bn);
    const int first = u.n * a.bn + half * 128;
    float m = neg_inf(), y = 0.0f;
    bool mine = false;
    auto mask = [&](float (&l)[64], int c) {  // words that there are not are out of the running
      const int w0 = first + 64 * c;
      if (w0 + 64 > end) {
#pragma unroll
        for (int i = 0; i < 64; i++)
          if (w0 + i >= end) l[i] = neg_inf();
      }
    };
    auto find = [&](const float (&l)[64], int c) {
      const int w0 = first + 64 * c;
      if (label >= w0 && label < min(w0 + 64, end)) {
        mine = true;
#pragma unroll
        for (int i = 0; i < 64; i++)
          if (label == w0 + i) y = l[i];
      }
#pragma unroll
      for (int i = 0; i < 64; i++) m = fmaxf(m, l[i]);
    };
    float by = 0.0f;
    bool keep = false;
    int p = 0;
    pair_t sum = pair(0.0f, 0.0f);
    auto add_up = [&](const float (&l)[64], int c) {
      const int x = first + 64 * c - p * a.piece;
      if (KEEP && CG == 2 && keep) reuse();
#pragma unroll
      for (int v = 0; v < 8; v++) {
        uint32_t code[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const pair_t s = mul2(add2(pair(l[8 * v + 2 * i], l[8 * v + 2 * i + 1]), pair(-by, -by)), pair(kLog2e, kLog2e));
          sum = add2(sum, ex2_2(s));
          if constexpr (KEEP) code[i] = keep2<DT>(s);
        }
        if constexpr (KEEP) {
          if (!keep) continue;
          const uint4 codes = make_uint4(code[0], code[1], code[2], code[3]);
          if constexpr (CG == 2) {
            put_smem(staged(out, lane, v), codes);
          } else if (r < live && x + 8 * v < end - p * a.piece) {  // (few rows, and tiles of any multiple of 32 words)
            reinterpret_cast<uint4*>(static_cast<char*>(a.g) + (((int64_t)p * a.cap + r) * a.piece + x) * 2)[v] = codes;
          }
        }
      }
      if (KEEP && CG == 2 && keep) send(x, (int)(p * a.cap) + r0);
    };
    auto begin_sum = [&]() {
      by = shift_of(m);
      keep = KEEP && first < a.keep;
      p = keep ? first / a.piece : 0;
    };
    if constexpr (LONG) {
      const bool one = first < end, two = first + 64 < end;
      if (one) mask(sums[0], 0), find(sums[0], 0);
      if (two) mask(sums[1], 1), find(sums[1], 1);
      begin_sum();
      if (one) add_up(sums[0], 0);
      if (two) add_up(sums[1], 1);
    } else {
      float l[64];
      auto logits = [&](int c) {
        tmem_load(tmem + (uint32_t)(64 * c), l);
        mask(l, c);
      };
      for (int c = 0; c < 2 && first + 64 * c < end; c++) {
        logits(c);
        find(l, c);
      }
      // (tensor memory is read a second time: that costs less than adjusting sums and what
      // is kept to a maximum that grows)
      begin_sum();
      for (int c = 0; c < 2 && first + 64 * c < end; c++) {
        logits(c);
        add_up(l, c);
      }
    }
    const float s = sum.x + sum.y;
    if (r < live) {
      a.parts[(int64_t)r * a.n_parts + u.n * 2 + half] = make_float2(m, s);
      if (mine) a.label_logit[r] = y;
    }
  } else if constexpr (JOB == GRAD) {
    const bool on = r < live;
    const int label = on ? a.label[r] : -1;
    const float2 st = on ? a.stats[r] : make_float2(0.0f, 0.0f);
    const float w = on ? a.weight[r] * a.scale[0] : 0.0f;
    auto quarter_of = [&](int c) {  // 32 words, in f
      const int c0 = u.n * kN + half * 128 + 32 * c, w0 = a.v0 + c0;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const pair_t x = add2(pair(f[i], f[i + 1]), pair(-st.x, -st.x));
        const pair_t p = ex2_2(fma2(x, pair(kLog2e, kLog2e), pair(-st.y, -st.y)));
        f[i] = p.x;
        f[i + 1] = p.y;
      }
#pragma unroll
      for (int i = 0; i < 32; i++) f[i] *= w;
      if ((uint32_t)(label - w0) < 32u) {
        float g = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i++)
          if (label == w0 + i) g = f[i] -= w;
        a.left[r] = g - rounded<DT>(g);
      }
      if (!on || w0 + 32 > a.V) {
#pragma unroll
        for (int i = 0; i < 32; i++)
          if (!on || w0 + i >= a.V) f[i] = 0.0f;
      }
      if (!(c & 1)) reuse();
      stage32<DT>(out, lane, c & 1, f);
      if (c & 1) send(c0 - 32, (int)a.g0 + r0);
    };
    if constexpr (LONG) {
#pragma unroll
      for (int c = 0; c < 4; c++) {
#pragma unroll
        for (int i = 0; i < 32; i++) f[i] = sums[c / 2][32 * (c % 2) + i];
        quarter_of(c);
      }
    } else {
      for (int c = 0; c < 4; c++) {
        fetch(c);
        quarter_of(c);
      }
    }
  } else {
    const float un = a.scale[1];
    const int at = half * 32 * kM + quarter * 32 + lane;  // of the row's first columns in a tile's sums
    float4* const chains = reinterpret_cast<float4*>(u.part >= 0 ? Work<BACK, CG>::part_at(a, u.dw, u.part, rank)
                                                                 : Work<BACK, CG>::chains_at(a, me, rank)) + at;
    auto fetch_sum = [&](int c) {  // of all chains so far
      fetch(c);
      if (!begin) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float4 o = chains[(c * 8 + j) * kM];
          f[4 * j] += o.x; f[4 * j + 1] += o.y; f[4 * j + 2] += o.z; f[4 * j + 3] += o.w;
        }
      }
    };
    if (u.part >= 0 || !end) {
      const bool on = u.dw || r < live;
      for (int c = 0; c < 4; c++) {
        fetch_sum(c);
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (on) chains[(c * 8 + j) * kM] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
      }
    } else if (!u.dw) {
      const bool on = r < live;
      float4* sums = reinterpret_cast<float4*>(a.acc + ((int64_t)u.tile * CG + rank) * (int64_t)kTileFloats) + at;
      for (int c = 0; c < 4; c++) {
        fetch_sum(c);
        const int d0 = u.n * kN + half * 128 + 32 * c;
        if (!a.first) {
#pragma unroll
          for (int j = 0; j < 8; j++) {
            const float4 o = sums[(c * 8 + j) * kM];
            f[4 * j] += o.x; f[4 * j + 1] += o.y; f[4 * j + 2] += o.z; f[4 * j + 3] += o.w;
          }
        }
        if (!a.last) {
#pragma unroll
          for (int j = 0; j < 8; j++)
            sums[(c * 8 + j) * kM] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
        } else if (on) {
          typename Elem<DT>::T* to = static_cast<typename Elem<DT>::T*>(a.d_hidden) + (int64_t)a.map[r] * a.dh_stride + d0;
#pragma unroll
          for (int j = 0; j < 4; j++)
            if (d0 + 8 * j < a.D) {
              float g[8];
#pragma unroll
              for (int i = 0; i < 8; i++) g[i] = f[8 * j + i];
              add_left<DT>(a, r, d0 + 8 * j, g);
#pragma unroll
              for (int i = 0; i < 8; i++) g[i] *= un;
              reinterpret_cast<uint4*>(to)[j] = Elem<DT>::pack(g);
            }
        }
      }
    } else {
      auto finish = [&](auto get) {
        for (int c = 0; c < 4; c++) {
          get(c);
#pragma unroll
          for (int i = 0; i < 32; i++) f[i] *= un;
          if (!(c & 1)) reuse();
          stage32<DT>(out, lane, c & 1, f);
          if (c & 1) send(u.n * kN + half * 128 + 32 * (c - 1), a.v0 + r0);
        }
      };
      // (in one loop the tiles of few rows, which are epilogue for the most part, took 4 % longer)
      if (begin) finish(fetch);
      else finish(fetch_sum);
    }
  }
}

// Warp 0 copies tiles to shared memory, warp 1 (of a pair's first CTA) issues the products,
// warp 2 allocates tensor memory, warps 4 to 11 are the epilogue: two accumulators let it
// work on one tile during the products of the next.  Cycles of a loss of 9728 x 32000: with a
// dim of 1280 757 K, 831 K where the logits are kept (640 K at the tensor cores' full rate), of 2048
// 1152 K and 1260 K (1024 K); each 256 of dim are 132 to 137 K (128 K), the rest is the epilogue in the
// way of the products, and all of it below a dim of 512.  The time of large calls is that of the clock,
// which the power limit sets: 16384 x 32000 x 2048 in 1.12 ms (1.92 PFLOP/s) alone, 4.2 to 4.3 ms with both
// gradients.  Tiles of one CTA alone took 10 % more.
template <int JOB, int DT, int CG, bool KEEP, bool LONG>
__global__ __launch_bounds__(kThreads, 1) void product(const __grid_constant__ CUtensorMap map_a,
                                                       const __grid_constant__ CUtensorMap map_b,
                                                       const __grid_constant__ CUtensorMap map_wa,  // dW's operands
                                                       const __grid_constant__ CUtensorMap map_wb,
                                                       const __grid_constant__ CUtensorMap map_out,
                                                       const CeArgs a) {
  using S = Shape<CG>;
  constexpr int kMax = S::kMaxStages;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * kMax + 5];
  __shared__ uint32_t tmem_at;
  __shared__ volatile uint32_t gone;
  const uint32_t buf = (smem_at(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  auto full = [&](int s) { return smem_at(&bars[s]); };  // (of a pair: the first CTA's counts for both)
  auto free_ = [&](int s) { return smem_at(&bars[kMax + s]); };
  auto ready = [&](int s) { return smem_at(&bars[2 * kMax + s]); };
  auto taken = [&](int s) { return smem_at(&bars[2 * kMax + 2 + s]); };  // (the same)
  auto meet = [&]() {
    fence_before();
    if constexpr (CG == 2) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    fence_after();
  };
  if (warp == 0 && lane == 0) {
    prefetch_map(&map_a);
    prefetch_map(&map_b);
    if (JOB == BACK) {
      prefetch_map(&map_wa);
      prefetch_map(&map_wb);
    }
    gone = 0u;
    for (int s = 0; s < kMax; s++) {
      bar_init(full(s), 1);
      bar_init(free_(s), 1);
    }
    for (int s = 0; s < 2; s++) {
      bar_init(ready(s), 1);
      bar_init(taken(s), kEpiWarps * CG);
    }
#ifdef SCAPE_DEBUG_CHECKS
    bar_init(smem_at(&bars[2 * kMax + 4]), 1);
#endif
    bar_init_fence();
  }
  __syncwarp();
  if (warp == 2) tmem_alloc<CG>(smem_at(&tmem_at), 512);
  meet();
  const uint32_t tmem = tmem_at;
  grid_launch_dependents();
  const int cols = JOB == BACK ? kN : a.bn;  // of a tile
  const uint32_t bytes_a = (JOB == BACK ? kM : a.bm) * kK * 2, bytes_b = cols / CG * kK * 2, stage = bytes_a + bytes_b;
  const int stages = min(kMax, (int)(kRing / stage));
  // Few rows: the first weights are on their way while the rows are still being taken
  // (with at most one row of tiles, unit i is tile i).
  int early = 0;
  if (JOB == LOSS && CG == 1 && warp == 0 && lane == 0 && a.early && blockIdx.x * cols < a.V)
    for (; early < min(stages, (a.D + kK - 1) / kK); early++) {
      bar_expect(full(early), stage);
      load_box<CG>(buf + early * stage + bytes_a, &map_b, early * kK, blockIdx.x * cols, full(early));
    }
  grid_dependency_wait();
  const int live = *a.live;
  const Work<JOB, CG> work(a, live);
  Unit t;
  __syncwarp();
  if (warp < 4) {
    if constexpr (LONG) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOthers));
    if (warp == 0 && lane == 0) {
      if (live == 0)  // no row after all: the stages are completed and left
        for (int s = 0; s < early; s++) {
          load_box<CG>(buf + s * stage, &map_a, 0, 0, full(s));
          bar_wait(full(s), 0, &gone);
        }
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int j = 0; ok && work.get(first, step, j, t); j++) {
        const int m0 = t.m * S::kRows + rank * kM, n0 = t.n * cols + rank * (cols / CG);
        for (int k = t.k0; k < t.k1; k++) {
          const bool begun = early > 0;
          if (!begun && !(ok = bar_wait(free_(s), ph ^ 1u, &gone))) break;
          const uint32_t sa = buf + s * stage, sb = sa + bytes_a;
          const uint32_t bar = CG == 2 ? bar_of(full(s), 0) : full(s);
          if (rank == 0 && !begun) bar_expect(full(s), ((t.dw ? kM : a.bm) * kK * 2 + bytes_b) * CG);
          if (JOB != BACK) {
            load_box<CG>(sa, &map_a, k * kK, m0, bar);
            if (begun) early--;
            else load_box<CG>(sb, &map_b, k * kK, a.v0 + n0, bar);
          } else if (!t.dw) {
            load_box<CG>(sa, &map_a, k * kK, (int)a.g0 + m0, bar);
#pragma unroll
            for (int i = 0; i < S::kCols / 64; i++) load_box<CG>(sb + i * 8192, &map_b, n0 + 64 * i, a.v0 + k * kK, bar);
          } else {
#pragma unroll
            for (int i = 0; i < kM / 64; i++) load_box<CG>(sa + i * 8192, &map_wa, m0 + 64 * i, (int)a.g0 + k * kK, bar);
#pragma unroll
            for (int i = 0; i < S::kCols / 64; i++) load_box<CG>(sb + i * 8192, &map_wb, n0 + 64 * i, k * kK, bar);
          }
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      int s = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int j = 0; ok && work.get(first, step, j, t); j++) {
        if (t.k0 >= t.k1) continue;  // nothing to multiply: no accumulator
        const bool across_a = JOB == BACK && t.dw;
        const uint32_t kind = product_of(DT == SCAPE_BF16, across_a, JOB == BACK, S::kRows, cols);
        for (int k = t.k0; ok && k < t.k1;) {
          const int acc = n & 1;
          if (!(ok = bar_wait(taken(acc), ((n >> 1) & 1) ^ 1, &gone))) break;
          n++;
          fence_after();
          const uint32_t d = tmem + acc * kN;
          const int k0 = k, k1 = chain_end<JOB, LONG>(t, k);
          for (; k < k1; k++) {
#ifdef SCAPE_DEBUG_CHECKS
            if (a.lost == 1 + JOB && blockIdx.x == 0 && !(ok = bar_wait(smem_at(&bars[2 * kMax + 4]), 0, &gone))) break;
#endif
            if (!(ok = bar_wait(full(s), ph, &gone))) break;
            fence_after();
            const uint32_t sa = buf + s * stage, sb = sa + bytes_a;
            // 16 elements of K: 32 bytes along a row, or 16 rows of 128 bytes
            const uint64_t oa = across_a ? operand(sa, 8192, 1024) : operand(sa, 16, 1024);
            const uint64_t ob = JOB == BACK ? operand(sb, 8192, 1024) : operand(sb, 16, 1024);
#pragma unroll
            for (int i = 0; i < kK / 16; i++)
              mma<CG>(d, oa + i * (across_a ? 128 : 2), ob + i * (JOB == BACK ? 128 : 2), kind, k > k0 || i > 0);
            commit<CG>(free_(s));
            if (++s == stages) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (ok) commit<CG>(ready(acc));
        }
      }
    }
  } else {
    if constexpr (LONG) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpilogue));
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    int n = 0;
    const uint32_t out = buf + kRing + (warp - 4) * kOutBytes;
    bool ok = true;
    float sums[2][LONG ? 64 : 1];
    for (int j = 0; ok && work.get(first, step, j, t); j++) {
      const bool empty = t.k0 >= t.k1;
      for (int k = t.k0, k1;; k = k1) {
        k1 = chain_end<JOB, LONG>(t, k);
        const int acc = n & 1;
        if (!empty) {
          if (!(ok = bar_wait(ready(acc), (n >> 1) & 1, &gone))) break;
          fence_after();
        }
        __syncwarp();
        const uint32_t at = tmem + acc * kN + half * 128 + ((uint32_t)(quarter * 32) << 16);
        auto finish = [&]() {
          epilogue<JOB, DT, CG, KEEP, LONG>(a, &map_out, t, live, first, (int)rank, half, quarter, lane, at, empty, k == t.k0,
                                            k1 == t.k1, out, sums);
        };
        if constexpr (LONG) {
          if (k == t.k0) {
            tmem_load(at, sums[0]);
            tmem_load(at + 64, sums[1]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; c++) {
              float f[32];
              tmem_load(at + 32 * c, f);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float *x = &sums[c / 2][32 * (c % 2) + i], *y = x + 1;
                const pair_t both = add2(pair(*x, *y), pair(f[i], f[i + 1]));
                *x = both.x;
                *y = both.y;
              }
            }
          }
        } else {
          finish();
        }
        if (!empty) {
          fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2) bar_arrive_at(bar_of(taken(acc), 0));
            else bar_arrive(taken(acc));
          }
          n++;
        }
        if (k1 == t.k1) {
          if constexpr (LONG) finish();
          break;
        }
      }
    }
    if (lane == 0) store_done();
  }
  // A wait ran out (never in a correct run): what is still being copied or multiplied ends
  // meanwhile.  All roles have ended, so nothing is started any more; a CTA whose own waits all
  // came true has nothing under way (its epilogue saw all of its products), and what its peer
  // has, the peer waits for.
  __syncwarp();
  __syncthreads();
  if (gone && threadIdx.x == 0) {
    const uint64_t began = now_ns();
    while (now_ns() - began < kDrainNs) {
    }
  }
  __syncwarp();
  meet();  // (neither CTA of a pair leaves while the other one's products and arrivals may still reach it)
  if (gone) {  // the losses say so, and the gradients (join_parts)
    if (threadIdx.x == 0) *a.status = 1u;
    for (int64_t i = threadIdx.x; i < a.rows; i += kThreads) a.loss[i] = __uint_as_float(0x7FFFFFFFu);
  }
  __syncwarp();
  if (warp == 2) tmem_free<CG>(tmem, 512);
}

// ---- rows -------------------------------------------------------------------------

struct RowsArgs {
  const int64_t* labels;
  const float* row_weight;
  int64_t rows, chunk;  // chunk: rows of a CTA
  int V;
  const char* hidden;
  int64_t stride, bytes;  // of a row, in bytes
  char* d_hidden;         // or NULL
  int64_t dh_stride;      // bytes
  int32_t* map;
  int32_t* label;
  float* weight;
  char* together;         // cap x D
  int32_t* live;
  float* scale;
  uint32_t* status;
  float* loss;
  uint32_t* bad;
  float target;  // what the largest weight becomes
};

// The rows with a term, together and in their order.  Each CTA takes a chunk of the
// rows and counts those in front of it by itself: at most 512 CTAs read all labels,
// which costs less than a second kernel.  The rows without a term get their loss and
// gradient of 0.  (One CTA that numbers the rows took 33 us for 16384 of them, and a second
// kernel 20 us to copy them; this one copies them in 31 us, 4096 rows in 9.)
constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32, kMaxRowCtas = 512;
__global__ __launch_bounds__(kRowThreads) void take_rows(const RowsArgs a) {
  __shared__ uint32_t scan[kRowWarps + 1];
  __shared__ uint32_t ubuf[32];
  __shared__ float fbuf[32];
  __shared__ int64_t place[kRowThreads];
  const int tid = threadIdx.x;
  const int64_t begin = blockIdx.x * a.chunk, end = min(a.rows, begin + a.chunk);
  float top = 0.0f;
  auto look = [&](int64_t r, int64_t& y, float& w) {
    y = a.labels[r];
    w = a.row_weight ? a.row_weight[r] : 1.0f;
    const bool on = y >= 0 && y < a.V && w != 0.0f;
    if (on && fabsf(w) < INFINITY) top = fmaxf(top, fabsf(w));
    return on;
  };
  uint32_t before = 0, n_bad = 0;
  int64_t y;
  float w;
  grid_dependency_wait();
#pragma unroll 8
  for (int64_t r = tid; r < begin; r += kRowThreads) before += look(r, y, w);
  int64_t at = cta_sum(before, ubuf);  // (rows < 2^24)
  grid_launch_dependents();  // (not ahead of the wait: LOSS loads weights ahead of its own)
  const uint32_t vecs = (uint32_t)(a.bytes / 16);  // (up to 8192, of 512 rows)
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int64_t r0 = begin; r0 < end; r0 += kRowThreads) {
    const int64_t r = r0 + tid;
    const bool in = r < end, on = in && look(r, y, w);
    uint32_t all;
    const uint32_t rank = block_incl_scan<kRowThreads>(on, scan, &all) - on;
    if (on) {
      a.map[at + rank] = (int32_t)r;
      a.label[at + rank] = (int32_t)y;
      a.weight[at + rank] = w;
    } else if (in) {
      a.loss[r] = 0.0f;
      n_bad += y >= a.V && w != 0.0f;
    }
    place[tid] = on ? at + rank : -1;
    __syncthreads();
    const int n = (int)min((int64_t)kRowThreads, end - r0);
#pragma unroll 4
    for (uint32_t x = tid; x < (uint32_t)n * vecs; x += kRowThreads) {
      const uint32_t i = x / vecs, v = x - i * vecs;
      const int64_t p = place[i];
      if (p >= 0)
        reinterpret_cast<uint4*>(a.together + p * a.bytes)[v] =
            ld_row_u4(reinterpret_cast<const uint4*>(a.hidden + (r0 + i) * a.stride) + v);
      else if (a.d_hidden)
        reinterpret_cast<uint4*>(a.d_hidden + (r0 + i) * a.dh_stride)[v] = zero;
    }
    __syncthreads();
    at += all;
  }
  n_bad = cta_sum(n_bad, ubuf);
  if (tid == 0 && a.bad && n_bad) atomicAdd(a.bad, n_bad);
  if (blockIdx.x + 1 < gridDim.x) return;
  // the last CTA has seen every row.  Rows of 0 behind the last one, to a multiple of 64:
  // the product of dW adds them up, too
  if (a.d_hidden)
    for (int64_t i = at * vecs + tid; i < (at + 63) / 64 * 64 * vecs; i += kRowThreads)
      reinterpret_cast<uint4*>(a.together)[i] = zero;
  top = cta_max(top, fbuf);
  if (tid == 0) {
    *a.live = (int32_t)at;
    *a.status = 0u;
    float s = 1.0f;
    const int e = (int)((__float_as_uint(top) >> 23) & 0xFF);
    if (e >= 30) s = fmaxf(a.target / top, 0x1p-126f);  // (its reciprocal is finite; a bf16 weight becomes 4 at most)
    else if (e > 0) s = a.target * 0x1p97f;             // (0: no weight or a denormal one)
    a.scale[0] = s;
    a.scale[1] = 1.0f / s;
  }
}

// A warp a row: maximum and sum of its parts, and its loss.
__global__ __launch_bounds__(256) void row_losses(const CeArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, r = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= *a.live) return;
  auto join = [](float2 p, float2 q) {
    const float m = fmaxf(p.x, q.x), by = shift_of(m);
    return make_float2(m, p.y * ex2((p.x - by) * kLog2e) + q.y * ex2((q.x - by) * kLog2e));
  };
  float2 p = make_float2(neg_inf(), 0.0f);
#pragma unroll 8
  for (int i = lane; i < a.n_parts; i += 32) p = join(p, a.parts[(int64_t)r * a.n_parts + i]);
#pragma unroll
  for (int o = 16; o; o >>= 1)
    p = join(p, make_float2(__shfl_xor_sync(kFull, p.x, o), __shfl_xor_sync(kFull, p.y, o)));
  if (lane == 0) {
    a.stats[r] = make_float2(p.x, log2f(p.y));
    const float loss = a.weight[r] * ((p.x - a.label_logit[r]) + logf(p.y));
    a.loss[a.map[r]] = *a.status ? __uint_as_float(0x7FFFFFFFu) : loss;
  }
}

// G of a piece in the place of what was kept of its logits, s:
//   p = 2^(s + (m_part - m) log2e - log2 sum),  G = w (p - [label]), w scaled
// A warp has a run of a row, six vectors a lane.  Bound by HBM and by the arithmetic of the codes:
// 4096 x 50257 in 135 us (6.1 TB/s), with four vectors and four CTAs an SM 139, with five 155.
template <int DT>
__global__ __launch_bounds__(256, 3) void grad_kept(const CeArgs a) {
  using E = Elem<DT>;
  constexpr int kVecs = 6, kRun = 32 * kVecs;
  grid_launch_dependents();
  grid_dependency_wait();
  const int live = *a.live, lane = threadIdx.x & 31;
  const int64_t rows = up_div(live, kK) * kK;                     // (as many as the sums of dW take: those of dH
                                                                  // that have no row are not looked at)
  const int vecs = a.piece / 8, runs = (vecs + kRun - 1) / kRun;  // (beside the last word, too)
  const float scale = a.scale[0];
  for (int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); item < rows * runs; item += (int64_t)gridDim.x * 8) {
    const int r = (int)(item / runs), v0 = (int)(item - (int64_t)r * runs) * kRun + lane;
    uint4* row = reinterpret_cast<uint4*>(static_cast<char*>(a.g) + (a.g0 + r) * a.piece * 2);
    if (r >= live) {
#pragma unroll
      for (int i = 0; i < kVecs; i++)
        if (v0 + 32 * i < vecs) row[v0 + 32 * i] = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 e[kVecs];
    float m[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; i++) {
      const int v = v0 + 32 * i, word = a.v0 + 8 * v;
      m[i] = neg_inf();
      if (v < vecs && word < a.V) {
        e[i] = ld_row_u4(row + v);
        const int tile = word / a.bn;
        m[i] = a.parts[(int64_t)r * a.n_parts + 2 * tile + (word - tile * a.bn >= 128)].x;
      }
    }
    const float2 st = a.stats[r];
    const float w = a.weight[r] * scale;
    const int label = a.label[r] - a.v0;
#pragma unroll
    for (int i = 0; i < kVecs; i++) {
      const int v = v0 + 32 * i, left = a.V - (a.v0 + 8 * v);  // words from here on
      if (v >= vecs) break;
      float x[8];
      if (left > 0) {
        kept8<DT>(e[i], __fmaf_rn(m[i] - st.x, kLog2e, -st.y), w, x);
        if (left < 8) {
#pragma unroll
          for (int j = 0; j < 8; j++)
            if (j >= left) x[j] = 0.0f;
        }
        if ((uint32_t)(label - 8 * v) < 8u) {
          const float g = w * (ex2(__fmaf_rn(a.label_logit[r] - st.x, kLog2e, -st.y)) - 1.0f);
          a.left[r] = g - rounded<DT>(g);
#pragma unroll
          for (int j = 0; j < 8; j++)
            if (label == 8 * v + j) x[j] = g;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] = 0.0f;
      }
      row[v] = E::pack(x);
    }
  }
}

// The parts of the split tiles, added up in order: a thread has eight columns of a row.
// Where a wait ran out, behind the last piece, all gradients become NaN.
template <int DT, int CG>
__global__ __launch_bounds__(256) void join_parts(const CeArgs a) {
  constexpr int kRows = Shape<CG>::kRows;
  grid_launch_dependents();
  grid_dependency_wait();
  if (*a.status) {
    if (!a.last) return;
    const int64_t vecs = a.D / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (a.rows + a.V) * vecs; i += (int64_t)gridDim.x * 256) {
      const int64_t row = i / vecs;
      char* to = row < a.rows ? static_cast<char*>(a.d_hidden) + row * a.dh_stride * 2
                              : static_cast<char*>(a.d_weight) + (row - a.rows) * a.dw_stride * 2;
      reinterpret_cast<uint4*>(to)[i - row * vecs] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
    }
    return;
  }
  const int live = *a.live;
  const Work<BACK, CG> work(a, live);
  const float un = a.scale[1];
  const int of_h = work.split_h > 1 ? work.h.count() : 0, tiles = of_h + work.rest();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)tiles * kRows * (kN / 8);
       i += (int64_t)gridDim.x * 256) {
    const int row = (int)(i % kM), j = (int)(i / kM % (kN / 8)), both = (int)(i / (kM * (kN / 8)));
    const int rank = both % CG;
    int t = both / CG;
    const bool dw = t >= of_h;
    if (dw) t -= of_h;
    const Tiles& all = dw ? work.w : work.h;
    const int tile = dw ? work.whole + t : t, step = dw ? work.rest() : of_h, parts = dw ? work.split_w : work.split_h;
    int m, n;
    all.place(tile, m, n);
    const int r = m * kRows + rank * kM + row, d = n * kN + 8 * j;
    if (d >= a.D || (dw ? a.v0 + r >= a.V : r >= live)) continue;
    float f[8] = {};
    auto add = [&](const float* sums) {
      const float4* q = reinterpret_cast<const float4*>(sums) + 2 * j * kM + row;
      const float4 x = q[0], y = q[kM];
      f[0] += x.x; f[1] += x.y; f[2] += x.z; f[3] += x.w;
      f[4] += y.x; f[5] += y.y; f[6] += y.z; f[7] += y.w;
    };
    for (int s = 0; s < parts; s++) add(Work<BACK, CG>::part_at(a, dw, s * step + t, rank));
    if (!dw) {
      float* acc = a.acc + ((int64_t)tile * CG + rank) * (int64_t)kTileFloats;
      if (!a.first) add(acc);
      if (!a.last) {
        float4* q = reinterpret_cast<float4*>(acc) + 2 * j * kM + row;
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[kM] = make_float4(f[4], f[5], f[6], f[7]);
        continue;
      }
    }
    if (!dw) add_left<DT>(a, r, d, f);
#pragma unroll
    for (int e = 0; e < 8; e++) f[e] *= un;
    typename Elem<DT>::T* out =
        dw ? static_cast<typename Elem<DT>::T*>(a.d_weight) + (int64_t)(a.v0 + r) * a.dw_stride + d
           : static_cast<typename Elem<DT>::T*>(a.d_hidden) + (int64_t)a.map[r] * a.dh_stride + d;
    *reinterpret_cast<uint4*>(out) = Elem<DT>::pack(f);
  }
}

// ---- host -------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static std::atomic<EncodeFn> cache{nullptr};
  EncodeFn fn = cache.load(std::memory_order_acquire);
  if (fn) return fn;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult st{};
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
      st != cudaDriverEntryPointSuccess)
    return nullptr;
  fn = reinterpret_cast<EncodeFn>(p);
  cache.store(fn, std::memory_order_release);
  return fn;
}

// Rows of "cols" 16-bit elements, "ld" apart; boxes of 64 columns and "box" rows.
bool encode(CUtensorMap* map, int dtype, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
  const cuuint32_t boxes[2] = {64, box}, steps[2] = {1, 1};
  const EncodeFn fn = encoder();
  return fn && fn(map, dtype == SCAPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                  const_cast<void*>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint64_t up(uint64_t x, uint64_t y) { return (x + y - 1) / y * y; }

// How a call is cut, by its sizes alone.
struct Cut {
  uint64_t cap = 0;     // rows, rounded up
  uint64_t bn = kN;     // words of a tile of LOSS
  uint64_t piece = 0;   // words of a piece
  uint64_t pieces = 0;
  uint64_t kept = 0;    // pieces that LOSS keeps
  uint64_t n_parts = 0;
};

// G takes at most this much, so that a gradient needs little memory beside its results:
// of a piece, and of all pieces that are there at once (kept ones; the others come one
// after the other).  Pieces of half and of twice the size: 16384 x 32000 in 4.44 and 4.28 ms
// instead of 4.10.
constexpr uint64_t kPieceBytes = 512ull << 20, kAllBytes = 1024ull << 20;

uint64_t ceil_div(uint64_t x, uint64_t y) { return (x + y - 1) / y; }

Cut cut_of(const scape_linear_ce_args* q, bool grad) {
  Cut c;
  // (whole tiles; of few rows as many as the sums over them take at a time)
  c.cap = q->rows <= kM ? up(std::max<uint64_t>(q->rows, 1), kK) : up(q->rows, Shape<2>::kRows);
  // Few rows: the weights' way to the CTAs is what takes time, and tiles of 256 words leave
  // CTAs without any.  The width that needs the fewest words a CTA, all rounds together
  // (32 for a tile's other costs).  16 rows, 32000 words: 224 a tile 30.7 us, 256 32.4, 112 35.2, 64 52.
  if (q->rows <= kM) {
    const uint64_t sms = (uint64_t)num_sms();
    uint64_t best = ~0ull;
    for (uint64_t n = kN; n >= 32; n -= 32) {
      const uint64_t words = ceil_div(ceil_div(q->vocab, n), sms) * (n + 32);
      if (words < best) {
        best = words;
        c.bn = n;
      }
    }
  }
  c.n_parts = 2 * ceil_div(q->vocab, c.bn);
  if (!grad) return c;
  const uint64_t tiles = ceil_div(q->vocab, kN);
  const uint64_t fit = std::max<uint64_t>(kPieceBytes / (c.cap * 2 * kN), 1);
  c.piece = ceil_div(tiles, ceil_div(tiles, fit)) * kN;
  c.pieces = ceil_div(tiles * kN, c.piece);
  // (a tile of another width may lie in two pieces)
  if (c.pieces == 1 || c.bn == (uint64_t)kN)
    c.kept = std::min(c.pieces, std::max<uint64_t>(kAllBytes / (c.cap * c.piece * 2), 1));
  return c;
}

struct Layout {
  uint64_t map, label, weight, logit, left, parts, stats, head, rows, g, acc, tail, bytes;
};

Layout layout_of(const scape_linear_ce_args* q, const Cut& c, bool grad) {
  Layout l{};
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t p = at;
    at += up(bytes, 256);
    return p;
  };
  l.head = take(64);
  l.map = take(c.cap * 4);
  l.label = take(c.cap * 4);
  l.weight = take(c.cap * 4);
  l.logit = take(c.cap * 4);
  l.left = take(c.cap * 4);
  l.stats = take(c.cap * 8);
  l.parts = take(c.n_parts * c.cap * 8);
  l.rows = take(c.cap * q->dim * 2);
  if (grad) {
    l.g = take(std::max<uint64_t>(c.kept, 1) * c.cap * c.piece * 2);
    if (c.pieces > 1) l.acc = take(ceil_div(c.cap, kM) * ceil_div(q->dim, kN) * kTileFloats * 4);
    l.tail = take(2 * kMaxParts * (uint64_t)num_sms() * kTileFloats * 4);
  }
  l.bytes = at;
  return l;
}

int check_sizes(const scape_linear_ce_args* q) {
  if (!q) return fail(SCAPE_EINVAL, "args is NULL");
  if (q->dtype != SCAPE_BF16 && q->dtype != SCAPE_F16)
    return fail(SCAPE_EINVAL, "dtype=%d: hidden states and weights are bf16 or fp16", q->dtype);
  if (q->rows >= (1ull << 24)) return fail(SCAPE_EINVAL, "rows must be < 2^24");
  if (q->vocab < 1 || q->vocab >= (1ull << 24))
    return fail(SCAPE_EINVAL, "vocab=%llu must be in [1, 2^24)", (unsigned long long)q->vocab);
  if (q->dim < 8 || q->dim % 8 || q->dim > 65536)
    return fail(SCAPE_EINVAL, "dim=%llu must be a multiple of 8 in [8, 65536]", (unsigned long long)q->dim);
  if (!q->d_hidden != !q->d_weight) return fail(SCAPE_EINVAL, "d_hidden and d_weight come together");
  return SCAPE_OK;
}

int check_matrix(const void* p, uint64_t stride, uint64_t dim, const char* name) {
  if (stride < dim || stride % 8 || stride >= (1ull << 32))
    return fail(SCAPE_EINVAL, "%s: the row stride must be a multiple of 8, >= dim and < 2^32", name);
  if (misaligned(p, 16)) return fail(SCAPE_EINVAL, "%s must be 16-byte aligned", name);
  return SCAPE_OK;
}

template <int JOB, int DT, int CG, bool KEEP, bool LONG>
cudaError_t launch_one(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mwa, const CUtensorMap& mwb,
                           const CUtensorMap& mo, const CeArgs& a, uint64_t tiles, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(product<JOB, DT, CG, KEEP, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    if (LONG) {  // (the epilogue would wait for registers that there are not)
      cudaFuncAttributes fa{};
      e = cudaFuncGetAttributes(&fa, product<JOB, DT, CG, KEEP, LONG>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs * kThreads < 128 * kRegsOthers + (kThreads - 128) * kRegsEpilogue) return cudaErrorInvalidConfiguration;
    }
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  unsigned grid = (unsigned)a.grid;  // (BACK divides its work by it)
  if (JOB != BACK) grid = (unsigned)std::min<uint64_t>(std::max<uint64_t>(tiles, 1), grid);
  return launch_clusters(product<JOB, DT, CG, KEEP, LONG>, grid * CG, kThreads, kSmem, CG, s, ma, mb, mwa, mwb, mo, a);
}

template <int JOB, int DT, int CG, bool KEEP = false>
cudaError_t launch_product(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mwa, const CUtensorMap& mwb,
                           const CUtensorMap& mo, const CeArgs& a, uint64_t tiles, cudaStream_t s) {
  if constexpr (JOB != BACK)
    if (a.D > kLongDim) return launch_one<JOB, DT, CG, KEEP, true>(ma, mb, mwa, mwb, mo, a, tiles, s);
  return launch_one<JOB, DT, CG, KEEP, false>(ma, mb, mwa, mwb, mo, a, tiles, s);
}

template <int DT, int CG>
int run(const scape_linear_ce_args* q, const Cut& c, const Layout& l, char* ws, cudaStream_t s) {
  const bool grad = q->d_hidden != nullptr;
  CeArgs a{};
  a.map = reinterpret_cast<int32_t*>(ws + l.map);
  a.label = reinterpret_cast<int32_t*>(ws + l.label);
  a.weight = reinterpret_cast<float*>(ws + l.weight);
  a.label_logit = reinterpret_cast<float*>(ws + l.logit);
  a.left = reinterpret_cast<float*>(ws + l.left);
  a.w = q->weight;
  a.w_stride = (int64_t)q->weight_stride;
  a.parts = reinterpret_cast<float2*>(ws + l.parts);
  a.stats = reinterpret_cast<float2*>(ws + l.stats);
  a.live = reinterpret_cast<int32_t*>(ws + l.head);
  a.scale = reinterpret_cast<float*>(ws + l.head + 8);
  a.status = reinterpret_cast<uint32_t*>(ws + l.head + 16);
  a.loss = q->loss;
  a.rows = (int64_t)q->rows;
  a.cap = (int64_t)c.cap;
  a.D = (int)q->dim;
  a.V = (int)q->vocab;
  constexpr int kRows = Shape<CG>::kRows;
  a.grid = num_sms() / CG;
#ifdef SCAPE_DEBUG_CHECKS
  const char* lost = std::getenv("SCAPE_TEST_LOST_WAIT");
  a.lost = lost ? std::atoi(lost) : 0;
#endif
  a.n_parts = (int)c.n_parts;
  char* rows = ws + l.rows;

  const uint64_t g_rows = std::max<uint64_t>(c.kept, 1) * c.cap;
  CUtensorMap along_h, along_w, across_h, across_w, along_g, across_g, piece_w, out_g, out_w;
  // (what is not copied of a tile's rows are rows that nobody reads)
  a.bm = CG == 1 ? (int)up(std::max<uint64_t>(q->rows, 1), 8) : kM;
  a.early = CG == 1;
  bool ok = encode(&along_h, q->dtype, rows, c.cap, q->dim, q->dim, (uint32_t)a.bm) &&
            encode(&along_w, q->dtype, q->weight, q->vocab, q->dim, q->weight_stride, (uint32_t)c.bn / CG);
  if (ok && grad)
    ok = encode(&piece_w, q->dtype, q->weight, q->vocab, q->dim, q->weight_stride, Shape<CG>::kCols) &&
         encode(&across_h, q->dtype, rows, c.cap, q->dim, q->dim, kK) &&
         encode(&across_w, q->dtype, q->weight, q->vocab, q->dim, q->weight_stride, kK) &&
         encode(&along_g, q->dtype, ws + l.g, g_rows, c.piece, c.piece, (uint32_t)a.bm) &&
         encode(&across_g, q->dtype, ws + l.g, g_rows, c.piece, c.piece, kK) &&
         encode(&out_g, q->dtype, ws + l.g, g_rows, c.piece, c.piece, 32) &&
         encode(&out_w, q->dtype, q->d_weight, q->vocab, q->dim, q->d_weight_stride, 32);
  if (!ok) return fail(SCAPE_ECUDA, "cuTensorMapEncodeTiled failed or is missing in the driver");

  RowsArgs ra{};
  ra.labels = q->labels;
  ra.row_weight = q->row_weight;
  ra.rows = a.rows;
  const uint64_t row_ctas = std::min<uint64_t>(std::max<uint64_t>(ceil_div(q->rows, 4), 1), kMaxRowCtas);
  ra.chunk = (int64_t)std::max<uint64_t>(ceil_div(q->rows, row_ctas), 1);
  ra.V = a.V;
  ra.hidden = static_cast<const char*>(q->hidden);
  ra.stride = (int64_t)q->hidden_stride * 2;
  ra.bytes = (int64_t)q->dim * 2;
  ra.d_hidden = static_cast<char*>(q->d_hidden);
  ra.dh_stride = (int64_t)q->d_hidden_stride * 2;
  ra.map = const_cast<int32_t*>(a.map);
  ra.label = const_cast<int32_t*>(a.label);
  ra.weight = const_cast<float*>(a.weight);
  ra.together = rows;
  ra.live = a.live;
  ra.scale = a.scale;
  ra.status = a.status;
  ra.loss = q->loss;
  ra.bad = q->bad_count;
  ra.target = DT == SCAPE_F16 ? 16384.0f : 1.0f;
  cudaError_t e = launch_behind(take_rows, (unsigned)std::max<uint64_t>(ceil_div(q->rows, (uint64_t)ra.chunk), 1),
                                kRowThreads, s, ra);
  if (e != cudaSuccess) return fail(SCAPE_ECUDA, "take_rows: %s", cudaGetErrorString(e));

  a.v0 = 0;
  a.vn = a.V;
  a.bn = (int)c.bn;
  a.g = ws + l.g;
  a.piece = (int)c.piece;
  a.keep = (int)std::min<uint64_t>(c.kept * c.piece, q->vocab);
  const uint64_t loss_tiles = ceil_div(q->rows, kRows) * ceil_div(q->vocab, c.bn);
  e = c.kept ? launch_product<LOSS, DT, CG, true>(along_h, along_w, along_h, along_w, out_g, a, loss_tiles, s)
             : launch_product<LOSS, DT, CG>(along_h, along_w, along_h, along_w, along_w, a, loss_tiles, s);
  if (e != cudaSuccess) return fail(SCAPE_ECUDA, "product (loss): %s", cudaGetErrorString(e));
  e = launch_behind(row_losses, (unsigned)ceil_div(std::max<uint64_t>(q->rows, 1), 8), 256, s, a);
  if (e != cudaSuccess) return fail(SCAPE_ECUDA, "row_losses: %s", cudaGetErrorString(e));
  if (!grad) return SCAPE_OK;

  a.acc = reinterpret_cast<float*>(ws + l.acc);
  a.tail = reinterpret_cast<float*>(ws + l.tail);
  a.d_hidden = q->d_hidden;
  a.dh_stride = (int64_t)q->d_hidden_stride;
  a.d_weight = q->d_weight;
  a.dw_stride = (int64_t)q->d_weight_stride;
  for (uint64_t p = 0; p < c.pieces; p++) {
    a.v0 = (int)(p * c.piece);
    a.vn = (int)std::min<uint64_t>(c.piece, q->vocab - p * c.piece);
    a.first = p == 0;
    a.last = p + 1 == c.pieces;
    if (p < c.kept) {
      a.g0 = (int64_t)(p * c.cap);
      a.bn = (int)c.bn;
      e = launch_behind(grad_kept<DT>, 3u * (unsigned)num_sms(), 256, s, a);
    } else {  // (the kept ones are done with)
      a.g0 = 0;
      a.bn = kN;
      e = launch_product<GRAD, DT, CG>(along_h, piece_w, along_h, piece_w, out_g, a, ceil_div(q->rows, kRows) * ceil_div(a.vn, kN), s);
    }
    if (e == cudaSuccess)
      e = launch_product<BACK, DT, CG>(along_g, across_w, across_g, across_h, out_w, a, 0, s);
    if (e == cudaSuccess) e = launch_behind(join_parts<DT, CG>, 4u * (unsigned)num_sms(), 256, s, a);
    if (e != cudaSuccess) return fail(SCAPE_ECUDA, "product (gradient): %s", cudaGetErrorString(e));
  }
  return SCAPE_OK;
}

}  // namespace
}  // namespace scape

SCAPE_API int scape_linear_ce_workspace(const scape_linear_ce_args* args, uint64_t* bytes) {
  using namespace scape;
  if (!bytes) return fail(SCAPE_EINVAL, "bytes is NULL");
  *bytes = 0;
  if (int rc = check_sizes(args)) return rc;
  const bool grad = args->d_hidden != nullptr;
  *bytes = layout_of(args, cut_of(args, grad), grad).bytes;
  return SCAPE_OK;
}

SCAPE_API int scape_linear_ce(const scape_linear_ce_args* args, void* workspace, uint64_t workspace_bytes,
                              void* stream) {
  using namespace scape;
  if (int rc = check_sizes(args)) return rc;
  const bool grad = args->d_hidden != nullptr;
  if (int rc = check_matrix(args->hidden, args->hidden_stride, args->dim, "hidden")) return rc;
  if (int rc = check_matrix(args->weight, args->weight_stride, args->dim, "weight")) return rc;
  if (!args->weight || (args->rows > 0 && (!args->hidden || !args->labels || !args->loss)))
    return fail(SCAPE_EINVAL, "hidden, weight, labels and loss are required");
  if (misaligned(args->labels, 8) || misaligned(args->row_weight, 4) || misaligned(args->loss, 4) ||
      misaligned(args->bad_count, 4))
    return fail(SCAPE_EINVAL, "a buffer is not aligned to its element size");
  if (grad) {
    if (int rc = check_matrix(args->d_hidden, args->d_hidden_stride, args->dim, "d_hidden")) return rc;
    if (int rc = check_matrix(args->d_weight, args->d_weight_stride, args->dim, "d_weight")) return rc;
    auto bytes = [&](uint64_t rows, uint64_t stride) { return rows ? ((rows - 1) * stride + args->dim) * 2 : 0; };
    const uint64_t h = bytes(args->rows, args->hidden_stride), w = bytes(args->vocab, args->weight_stride);
    const uint64_t dh = bytes(args->rows, args->d_hidden_stride), dw = bytes(args->vocab, args->d_weight_stride);
    if (ranges_meet(args->d_hidden, dh, args->hidden, h) || ranges_meet(args->d_hidden, dh, args->weight, w) ||
        ranges_meet(args->d_weight, dw, args->hidden, h) || ranges_meet(args->d_weight, dw, args->weight, w) ||
        ranges_meet(args->d_hidden, dh, args->d_weight, dw))
      return fail(SCAPE_EINVAL, "the gradients overlap each other or an input");
  }
  const Cut c = cut_of(args, grad);
  const Layout l = layout_of(args, c, grad);
  if (!workspace || misaligned(workspace, 256) || workspace_bytes < l.bytes)
    return fail(SCAPE_EINVAL, "workspace must be %llu bytes, 256-byte aligned", (unsigned long long)l.bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  // Pairs of CTAs, unless the rows of one are enough (dim 2048, 32000 words: 128 rows 34 us and 115 with gradients, in
  // pairs 38 and 121; 200 rows in pairs 38 and 131, in CTAs alone 42 and 140).
  if (args->rows <= (uint64_t)kM)
    return args->dtype == SCAPE_BF16 ? run<SCAPE_BF16, 1>(args, c, l, ws, s) : run<SCAPE_F16, 1>(args, c, l, ws, s);
  return args->dtype == SCAPE_BF16 ? run<SCAPE_BF16, 2>(args, c, l, ws, s) : run<SCAPE_F16, 2>(args, c, l, ws, s);
}
