// fp8_product.cuh -- the experts' products on FP8 operands with a power-of-two
// scale per 128 values, on CTA pairs (tcgen05 cta_group::2, block-scaled MMA).
//
//   rows   y[r] = sum_b 2^(sx[r,b] + sw[e,n/128,b]) sum_{k in block b} x[r,k] w[e,n,k]
//          for the rows r of expert e (forward; with the transposed weights the
//          gradient of the input)
//   wgrad  dw[e] = sum over the expert's blocks of 128 rows of dY^T X, each
//          operand scaled per (128 rows, column)
//   gated  act = f(gate) up with gate and up such products of the same rows with
//          two weights
//   gated backward  a product g, and from it g up f'(gate), g f(gate), f(gate) up
//   sum    the sum of two products, of other rows and weights each
//
// All have the weights' output rows on the accumulator's lanes (256 per pair
// tile, 128 per CTA; gated: 64 of either weight) and, on its columns, an
// expert's tokens (rows) or the weights' input columns (wgrad).  Tokens are the
// ragged side: an MMA may have any multiple of 32 columns, so an expert's tokens
// are cut into ceil(M / 224) tiles of equal width instead of being padded to
// 128.  224 is the widest that leaves room in TMEM for the scales beside two
// accumulators (2 x 224 + 32 <= 512 columns).
//
// The tensor cores multiply by the scales: each 128-wide K block is four MMAs
// (K = 32) that read one scale byte per row of A and of B from TMEM, where a
// 32-bit cell holds the bytes of four K blocks.  Up to four warps per CTA gather
// four blocks' bytes of the tile's rows at a time (a set), write them to a ring in
// shared memory apart from the operands', and the MMA thread copies a set to TMEM
// (tcgen05.cp) ahead of its MMAs.  Sets are counted from the tile's first K block
// (of either product), so rows need no alignment.
//
// A persistent pair walks the tiles.  Warp 0: TMA producer.  Warp 1: TMEM and,
// in the even CTA, the MMAs.  Then the epilogue's warps, overlapped with
// the next tile through the second accumulator, and the scales'.  The experts' rows
// are read from `offsets` on the device: every block sums the experts' tile
// counts before its first tile, so a call needs no host copy of the routing.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fp8_ptx.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "moe.h"
#include "muon.h"
#include "pair_math.cuh"

namespace muon {
namespace fp8 {

enum Mode { kRows, kWgrad, kGated, kGatedBackward, kSum };

constexpr int kTileM = 256;                       // pair tile: lanes of both accumulators
constexpr int kHalfM = 128;
constexpr int kGatedRows = kTileM / 2;            // gated: the lanes hold two weights' rows
constexpr int kBK = 128;                          // K block: one 128-byte swizzle row, one scale
constexpr int kABytes = kHalfM * kBK;             // 16 KB per CTA and stage
constexpr int kSetBlocks = 4;                     // K blocks per set of scales
constexpr int kScaleBytes = 512 + 1024;           // per set: 128 A cells, 256 B cells
constexpr int kMaxTokens = 224;                   // rows: widest token tile
constexpr int kWidthUnit = 32;                    // MMA columns come in multiples of this
constexpr int kGradN = 224;                       // wgrad: columns per tile (a multiple of 32), the
                                                  // last one's too: 0.4% idle at k = 8704, 4% at
                                                  // 4096, 9% at 1024, 39% at 272
constexpr int kTokenGroup = 8;                    // rows: token tiles that share a sweep over w
constexpr int kTmemCols = 512;
constexpr int kTmemScales = 448;
constexpr int kMaps = kMaxTokens / kWidthUnit;    // B boxes: half a width each

template <int MODE>
struct Layout {
  static constexpr bool GRAD = MODE == kWgrad;
  static constexpr int kEpiWarps = 4;                         // one per 32 lanes (eight: no faster)
  static constexpr int kScaleWarps = 4;                       // at most
  static constexpr int kSets = 8;                             // sets of scales in the ring
  static constexpr int kThreads = 32 * (2 + kEpiWarps + kScaleWarps);
  static constexpr int kAccCols = GRAD ? kGradN : kMaxTokens;
  static constexpr int kStages = GRAD || MODE == kGated ? 5 : 6;   // operand stages, at most
  // Gated: in tiles of 32 tokens an operand stage needs little beside w, and more
  // of them are in use.
  static constexpr int kFewStages = 8;
  static constexpr int kMaxStages = MODE == kGated ? kFewStages : kStages;
  static constexpr int kOutBufs = 2;                          // per epilogue warp
  static constexpr int kBBytes = (kAccCols / 2) * kBK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // One 32 x 32 chunk, FP32 or BF16.  (The backward pass of the gate works in one
  // FP32 buffer where others have two of BF16.)
  static constexpr int kOutBuf = GRAD || MODE == kGated ? 4096 : 2048;
  static constexpr int kFewBytes = kABytes + kWidthUnit / 2 * kBK;
  static_assert(kFewBytes % 1024 == 0 && kFewStages * kFewBytes <= kStages * kStageBytes || MODE != kGated,
                "the smaller stages");
  static constexpr int kScaleAt = kStages * kStageBytes;
  static constexpr int kOutAt = kScaleAt + kSets * kScaleBytes;
  static constexpr int kTableAt = kOutAt + kEpiWarps * kOutBufs * kOutBuf;
  static constexpr int kTableBytes = (kMoeMaxExperts + 4) * 4;
  static constexpr int kBarAt = kTableAt + 2 * kTableBytes;
  static constexpr int kSmem = kBarAt + 384 + 1024;
  static_assert(kBBytes % 1024 == 0 && kOutAt % 1024 == 0, "swizzle atoms");
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

struct Fp8Args {
  const uint8_t* a_scales;
  const uint8_t* b_scales;
  const uint8_t* a2_scales;   // gated: the second weight's; sum: the second product's
  const uint8_t* b2_scales;
  const int32_t* offsets;
  int32_t experts;
  int32_t n;            // rows of w / dw
  int32_t k;            // rows: contraction; wgrad: columns of dw
  int64_t rows;         // rows: rows of x and y; wgrad: columns of yt and xt
  int32_t n_blocks, k_blocks;
  int32_t tiles_m, tiles_n;
  __nv_bfloat16* y;           // gated: the activation, backward: or NULL
  __nv_bfloat16* gate;        // gated: out or NULL; backward: in
  __nv_bfloat16* up;
  __nv_bfloat16* grad_gate;   // gated backward
  __nv_bfloat16* grad_up;
  int32_t activation;
  int32_t stages;       // operand stages in use
  int32_t stage_bytes;  // gated: of each
  int32_t tile;         // gated: output rows of either weight per pair tile (a multiple of 16)
  int32_t scale_warps;  // scale warps in use (a divisor of kSets)
  int32_t accumulate;
  int* err;
};

template <int MODE>
struct Maps {
  CUtensorMap a;
  CUtensorMap b[kMaps];
  CUtensorMap out;            // wgrad: dw; gated and sum: the second weight
};
template <>
struct Maps<kSum> {
  CUtensorMap a;
  CUtensorMap b[kMaps];
  CUtensorMap out;
  CUtensorMap b2[kMaps];      // the second product's rows
};

struct Tile {
  int expert;
  int n0;               // first output row
  int c0;               // first token row (rows) or column of dw (wgrad)
  int cols;             // tokens or columns that exist
  int width;            // MMA columns (a multiple of kWidthUnit)
  int kb0, nkb;         // K blocks
  int last;             // K steps of 32 in the last one
};

// Output rows of w / dw per pair tile.
template <int MODE>
__device__ __forceinline__ int tile_rows(const Fp8Args& p) {
  return MODE == kGated ? p.tile : kTileM;
}

// first[e]: token tiles (rows) or row blocks (wgrad) before expert e;
// start[e]: its first row (rows) or how many rows it has (wgrad).
template <int MODE>
__device__ __forceinline__ bool decode(const Fp8Args& p, const int32_t* first, const int32_t* start,
                                       uint32_t t, Tile& o) {
  constexpr bool GRAD = MODE == kWgrad;
  const uint32_t tiles_m = p.tiles_m;
  if (GRAD) {
    const uint32_t per = tiles_m * p.tiles_n;
    o.expert = static_cast<int>(t / per);
    if (o.expert >= p.experts) return false;
    const uint32_t l = t - o.expert * per;
    // Along a row of tiles first: the pairs running at one time then write
    // whole rows of dw.
    const uint32_t tm = l / p.tiles_n;
    o.n0 = static_cast<int>(tm) * tile_rows<MODE>(p);
    o.c0 = static_cast<int>(l - tm * p.tiles_n) * kGradN;
    o.cols = min(kGradN, p.k - o.c0);
    o.width = kGradN;
    o.kb0 = first[o.expert];
    o.nkb = first[o.expert + 1] - o.kb0;
    // Columns past the next multiple of 32 rows were never written.
    o.last = min(4, (start[o.expert] - (o.nkb - 1) * kBK + 31) / 32);
    return true;
  }
  if (t >= first[p.experts] * tiles_m) return false;
  const int g = static_cast<int>(t / tiles_m);
  int lo = 0, hi = p.experts;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= g) lo = mid; else hi = mid;
  }
  // Within an expert: groups of kTokenGroup token tiles sweep over w
  // together, so that w is read from HBM once per group.
  const int tiles = first[lo + 1] - first[lo];
  const uint32_t l = t - first[lo] * tiles_m;
  const uint32_t group = l / (kTokenGroup * tiles_m);
  const uint32_t r = l - group * kTokenGroup * tiles_m;
  const uint32_t in_group = min(kTokenGroup, tiles - static_cast<int>(group) * kTokenGroup);
  const uint32_t tm = r / in_group;
  const int i = static_cast<int>(group * kTokenGroup + (r - tm * in_group));
  const int m = start[lo + 1] - start[lo];
  o.expert = lo;
  o.n0 = static_cast<int>(tm) * tile_rows<MODE>(p);
  o.width = min(kMaxTokens, ((m + tiles - 1) / tiles + kWidthUnit - 1) / kWidthUnit * kWidthUnit);
  o.c0 = start[lo] + i * o.width;
  o.cols = min(o.width, m - i * o.width);
  o.kb0 = 0;
  o.nkb = p.k_blocks;
  o.last = (p.k - (o.nkb - 1) * kBK + 31) / 32;
  return true;
}

// Fills first[] and start[] (all threads, a few experts each).  Whatever offsets
// holds, first[] rises no further than the buffers reach (64-bit sums: falling
// offsets can count rows many times) and start[] stays within x and y.
template <int MODE>
__device__ __forceinline__ void scan_experts(const Fp8Args& p, int32_t* first, int32_t* start,
                                             int64_t* warp_total) {
  constexpr bool GRAD = MODE == kWgrad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kPer = kMoeMaxExperts / Layout<MODE>::kThreads + 1;   // and the end of the last
  int count[kPer];
  int64_t sum = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    count[i] = 0;
    if (e < p.experts) {
      const int a = p.offsets[e], b = p.offsets[e + 1];
      if (GRAD) {
        bad = bad || a < 0 || b < a;
        const int rows = a < 0 || b < a ? 0 : b - a;
        start[e] = rows;
        count[i] = rows / kBK + (rows % kBK != 0 ? 1 : 0);
      } else {
        const int top = static_cast<int>(p.rows);
        const int ca = min(max(a, 0), top), cb = min(max(b, ca), top);
        bad = bad || ca != a || cb != b;
        start[e] = ca;
        if (e == p.experts - 1) start[p.experts] = cb;
        count[i] = (cb - ca + kMaxTokens - 1) / kMaxTokens;
      }
    }
    sum += count[i];
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  int64_t at = incl - sum;
  for (int i = 0; i < warp; ++i) at += warp_total[i];
  const int64_t limit = GRAD ? p.rows / kBK : p.rows / kMaxTokens + p.experts;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e <= p.experts) {
      bad = bad || at > limit;
      first[e] = static_cast<int32_t>(min(at, limit));
    }
    at += count[i];
  }
  if (bad && blockIdx.x == 0) atomicOr(p.err, kDevErrIndex);
}

// A wait by a whole warp with one outcome: when the limit expires in some lanes
// only, all of them give up together (the warp stays converged for what follows).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  return __all_sync(0xffffffffu, ptx::mbar_wait_cluster(bar, parity, abort));
}

// All of the 64 threads of barrier `id` (1..15) meet; true if `ok` is in all.
__device__ __forceinline__ bool meet_all(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %1, 64, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void meet(int id) {
  asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(id) : "memory");
}

// Gate activations, two values at a time: f(x) = x s(u(x)) with s the logistic function,
// u = x (silu) or 2 sqrt(2 / pi) (x + 0.044715 x^3) (gelu, its tanh form), or max(x, 0);
// and f' = s + x s (1 - s) u'.  The exponential and the reciprocal are the
// approximate instructions (2^-22 and 2^-23): their result is rounded to BF16.  Past
// |x| = 64 the logistic function is 0 or 1 in FP32 and u' has no part in f', so that
// x^2 is taken no further there (0 x inf).  (One at a time takes half as many instructions
// again: 16381 x 6144 x 4096 forward 486 us instead of 480, calls one after another.)
template <int KIND, bool SLOPE>
__device__ __forceinline__ Pair activate(Pair x, Pair* slope) {
  if (KIND == MUON_GATE_RELU) {
    float v[2], d[2];
    split(x, v[0], v[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool off = v[i] <= 0.0f;                  // (a NaN stays)
      d[i] = off ? 0.0f : v[i] > 0.0f ? 1.0f : v[i];
      if (off) v[i] = 0.0f;
    }
    if (SLOPE) *slope = pair_of(d[0], d[1]);
    return pair_of(v[0], v[1]);
  }
  constexpr float kGelu = 1.5957691216057308f, kLog2e = 1.4426950408889634f;
  Pair q = 0, w;                                      // w: -u log2(e)
  if (KIND == MUON_GATE_GELU) {
    q = mul2(x, x);
    w = mul2(mul2(x, pair_of(-kGelu * kLog2e)), fma2(q, pair_of(0.044715f), pair_of(1.0f)));
  } else {
    w = mul2(x, pair_of(-kLog2e));
  }
  float a, b;
  split(w, a, b);
  split(add2(pair_of(exp2_near(a), exp2_near(b)), pair_of(1.0f)), a, b);
  const Pair s = pair_of(rcp_near(a), rcp_near(b)), f = mul2(x, s);
  if (SLOPE) {
    Pair rest = mul2(f, fma2(s, pair_of(-1.0f), pair_of(1.0f)));
    if (KIND == MUON_GATE_GELU) {
      split(q, a, b);
      q = pair_of(fminf(a, 4096.0f), fminf(b, 4096.0f));
      rest = mul2(rest, fma2(q, pair_of(kGelu * 0.134145f), pair_of(kGelu)));
    }
    *slope = add2(rest, s);
  }
  return f;
}

// Calls f with the activation as a constant: chosen once for many values.
template <typename F>
__device__ __forceinline__ void with_activation(int kind, F f) {
  if (kind == MUON_GATE_SILU)
    f(std::integral_constant<int, MUON_GATE_SILU>{});
  else if (kind == MUON_GATE_GELU)
    f(std::integral_constant<int, MUON_GATE_GELU>{});
  else
    f(std::integral_constant<int, MUON_GATE_RELU>{});
}

__device__ __forceinline__ uint32_t pack_bf16(Pair p) {
  float a, b;
  split(p, a, b);
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

__device__ __forceinline__ uint4 pack_bf16(const Pair (&v)[4]) {
  return make_uint4(pack_bf16(v[0]), pack_bf16(v[1]), pack_bf16(v[2]), pack_bf16(v[3]));
}

__device__ __forceinline__ Pair unpack_bf16(uint32_t w) {
  return pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ void unpack_bf16(const uint4& u, Pair (&v)[4]) {
  v[0] = unpack_bf16(u.x);
  v[1] = unpack_bf16(u.y);
  v[2] = unpack_bf16(u.z);
  v[3] = unpack_bf16(u.w);
}

// A warp's chunk of 32 lanes (output columns) x 32 tokens through shared memory,
// FP32: column c of token t is word 32 t + (c ^ 4 (t & 1)), so that stores by
// column and 16-byte loads by token both hit all banks.
__device__ __forceinline__ void put_chunk(float* buf, int lane, const uint32_t (&v)[32]) {
#pragma unroll
  for (int t = 0; t < 32; ++t) buf[t * 32 + (lane ^ ((t & 1) << 2))] = __uint_as_float(v[t]);
}

__device__ __forceinline__ void get_columns(const float* buf, int t, int c, Pair (&v)[4]) {
  const int at = t * 32 + (c ^ ((t & 1) << 2));
  const float4 a = *reinterpret_cast<const float4*>(buf + at);
  const float4 b = *reinterpret_cast<const float4*>(buf + (at ^ 4));
  v[0] = pair_of(a.x, a.y);
  v[1] = pair_of(a.z, a.w);
  v[2] = pair_of(b.x, b.y);
  v[3] = pair_of(b.z, b.w);
}

// Walks the sets of scales of a pair's tiles.
struct SetCursor {
  uint32_t t;
  Tile o;
  int kb;               // first K block of the set
  int half;             // sum: which of the two products
  bool live;

  template <int MODE>
  __device__ __forceinline__ void begin(const Fp8Args& p, const int32_t* first, const int32_t* start,
                                        uint32_t t0) {
    t = t0;
    kb = 0;
    half = 0;
    live = decode<MODE>(p, first, start, t, o);
  }
  // Leaves a tile without K blocks at once.
  template <int MODE>
  __device__ __forceinline__ void settle(const Fp8Args& p, const int32_t* first,
                                         const int32_t* start, int step) {
    while (live && kb >= o.nkb) {
      kb = 0;
      if (MODE == kSum && half == 0 && o.nkb > 0) {
        half = 1;
        return;
      }
      half = 0;
      t += step;
      live = decode<MODE>(p, first, start, t, o);
    }
  }
  // `sets` sets further.
  template <int MODE>
  __device__ __forceinline__ void advance(const Fp8Args& p, const int32_t* first,
                                          const int32_t* start, int step, int sets) {
    for (int i = 0; i < sets && live; ++i) {
      kb += kSetBlocks;
      settle<MODE>(p, first, start, step);
    }
  }
};

// Scale bytes of n K blocks (1..4, `step` apart) for C rows at offsets off[] of
// `base`, as the rows' cells, byte 0 first.  Only the loads that are needed, all
// in flight together, with one 32-bit offset per row: a warp by itself takes
// these at the pace of its instructions.
template <int C>
__device__ __forceinline__ void load_cells(const uint8_t* __restrict__ base, int64_t step, int n,
                                           const uint32_t (&off)[C], uint32_t* cells) {
  uint32_t raw[kSetBlocks][C];
#pragma unroll
  for (int i = 0; i < kSetBlocks; ++i) {
    if (i < n) {
      const uint8_t* at = base + i * step;
#pragma unroll
      for (int c = 0; c < C; ++c) raw[i][c] = __ldg(at + off[c]);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) raw[i][c] = 0u;
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
    cells[c] = raw[0][c] | (raw[1][c] << 8) | (raw[2][c] << 16) | (raw[3][c] << 24);
}

// This lane's cells of one set: rows lane + 32 i, four of A's, seven of B's.
// Rows past the tile's or the matrix's read its last one's scales: they touch
// no result that is written.
constexpr int kCells = 4 + kMaxTokens / 32;
static_assert(kGradN <= kMaxTokens && kMaxTokens <= 256, "B's cells");

template <int MODE>
__device__ __forceinline__ void load_set(const Fp8Args& p, const SetCursor& s, uint32_t rank,
                                         int lane, uint32_t (&cells)[kCells]) {
  const Tile& o = s.o;
  const int row_a = o.n0 + static_cast<int>(rank) * (tile_rows<MODE>(p) / 2);
  const int n = min(kSetBlocks, o.nkb - s.kb);
  constexpr int kB = kCells - 4;
  uint32_t off[kB];
  if (MODE == kWgrad) {
    const int64_t kb = o.kb0 + s.kb;
    uint32_t off_a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) off_a[i] = min(row_a + i * 32 + lane, p.n - 1);
#pragma unroll
    for (int i = 0; i < kB; ++i) off[i] = min(o.c0 + i * 32 + lane, p.k - 1);
    load_cells<4>(p.a_scales + kb * p.n, p.n, n, off_a, cells);
    load_cells<kB>(p.b_scales + kb * p.k, p.k, n, off, cells + 4);
  } else {
    const bool second = MODE == kSum && s.half != 0;
    const int64_t a_at = s.kb + static_cast<int64_t>(o.expert) * p.n_blocks * p.k_blocks;
    const uint8_t* a = (second ? p.a2_scales : p.a_scales) + a_at;
    const uint8_t* b = (second ? p.b2_scales : p.b_scales) + s.kb + static_cast<int64_t>(o.c0) * p.k_blocks;
    const uint8_t* a2 = MODE == kGated ? p.a2_scales + a_at : a;
    // The block of rows that these lanes' row of w is in: one for all, or (gated,
    // whose tiles may be narrower than a block) for each of the two rows of a lane.
    constexpr int kA = MODE == kGated ? 2 : 1;
    uint32_t off_a[kA];
#pragma unroll
    for (int i = 0; i < kA; ++i) {
      const int row = MODE == kGated ? min(row_a + min(lane + i * 32, p.tile / 2 - 1), p.n - 1) : row_a;
      off_a[i] = static_cast<uint32_t>(min(row / kBK, p.n_blocks - 1)) * static_cast<uint32_t>(p.k_blocks);
    }
#pragma unroll
    for (int i = 0; i < kB; ++i) off[i] = min(i * 32 + lane, o.cols - 1) * p.k_blocks;
    // Rows of a multiple of four blocks start on a word (the buffers are
    // 16-byte aligned): one load per row.
    if (p.k_blocks % kSetBlocks == 0) {
#pragma unroll
      for (int i = 0; i < kA; ++i) {
        cells[i] = __ldg(reinterpret_cast<const uint32_t*>(a + off_a[i]));
        if (MODE == kGated) cells[2 + i] = __ldg(reinterpret_cast<const uint32_t*>(a2 + off_a[i]));
      }
#pragma unroll
      for (int i = 0; i < kB; ++i) cells[4 + i] = __ldg(reinterpret_cast<const uint32_t*>(b + off[i]));
    } else {
      load_cells<kA>(a, 1, n, off_a, cells);
      if (MODE == kGated) load_cells<kA>(a2, 1, n, off_a, cells + 2);
      load_cells<kB>(b, 1, n, off, cells + 4);
    }
    // (gated: lanes 64 to 127 are the second weight's rows)
    if (MODE != kGated) cells[1] = cells[2] = cells[3] = cells[0];
  }
}

// What the gated products' epilogue warps work with.
struct Epilogue {
  const int32_t* first;
  const int32_t* start;
  uint8_t* out;             // chunks in shared memory
  uint32_t tmem;
  uint64_t* full;           // accumulators
  uint64_t* empty;
  volatile int* abort_flag;
  uint32_t rank;
  int pair, npairs;
  int quad, lane;           // lanes 32 quad .. 32 quad + 31 of the accumulator

  __device__ __forceinline__ void give_up(int* err) const {
    if (lane == 0) {
      *abort_flag = 1;
      atomicOr(err, kDevErrTimeout);
    }
  }
  // Every value of accumulator `acc` has been read into registers.
  __device__ __forceinline__ void hand_back(int acc) const {
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0)
      ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_addr(&empty[acc]), 0));
  }
};

// Gated: lanes 0 to 63 of a CTA's accumulator are 64 columns of gate, lanes 64 to
// 127 the same columns of up (fewer where the tile is narrower).  The warps of two quarters 64 lanes apart meet once per
// chunk of 32 tokens, and either takes half of the tokens.  With two
// buffers each, a warp is past the meeting for a chunk only when the other has
// read the one before, whose place the next chunk takes.
__device__ __forceinline__ void gated_epilogue(const Fp8Args& p, const Epilogue& e) {
  using L = Layout<kGated>;
  constexpr int kFloats = L::kOutBuf / 4;
  float* bufs = reinterpret_cast<float*>(e.out);
  const int cols = e.quad & 1, id = 1 + cols;
  float* mine = bufs + e.quad * 2 * kFloats;
  const float* gates = bufs + cols * 2 * kFloats;
  const float* ups = gates + 4 * kFloats;
  int acc = 0, at = 0;
  uint32_t phase = 0;
  Tile o;
  for (uint32_t t = e.pair; decode<kGated>(p, e.first, e.start, t, o); t += e.npairs) {
    // Both warps go on, or neither.
    if (!meet_all(id, warp_wait(&e.full[acc], phase, e.abort_flag))) {
      e.give_up(p.err);
      break;
    }
    ptx::tc_fence_after();
    const uint32_t taddr = e.tmem + (static_cast<uint32_t>(e.quad * 32) << 16) +
                           static_cast<uint32_t>(acc * L::kAccCols);
    const int in_tile = cols * 32 + (e.lane & 3) * 8;
    const int n = in_tile < p.tile / 2 ? o.n0 + static_cast<int>(e.rank) * (p.tile / 2) + in_tile : p.n;
    const int chunks = (o.cols + 31) / 32;
    for (int cb = 0; cb < chunks; ++cb) {
      uint32_t v[32];
      __syncwarp();
      ptx::tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(cb * 32), v);
      ptx::tmem_ld_wait();
      if (cb == chunks - 1) e.hand_back(acc);
      put_chunk(mine + at * kFloats, e.lane, v);
      meet(id);
      with_activation(p.activation, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tt = (e.quad >> 1) * 16 + i * 8 + (e.lane >> 2), tok = cb * 32 + tt;
          Pair g[4], u[4], a[4];
          get_columns(gates + at * kFloats, tt, (e.lane & 3) * 8, g);
          get_columns(ups + at * kFloats, tt, (e.lane & 3) * 8, u);
#pragma unroll
          for (int q = 0; q < 4; ++q) a[q] = mul2(activate<kind.value, false>(g[q], nullptr), u[q]);
          if (tok < o.cols && n < p.n) {
            const int64_t to = static_cast<int64_t>(o.c0 + tok) * p.n + n;
            if (p.gate != nullptr) {
              *reinterpret_cast<uint4*>(p.gate + to) = pack_bf16(g);
              *reinterpret_cast<uint4*>(p.up + to) = pack_bf16(u);
            }
            *reinterpret_cast<uint4*>(p.y + to) = pack_bf16(a);
          }
        }
      });
      at ^= 1;
    }
    acc ^= 1;
    if (acc == 0) phase ^= 1u;
  }
}

// Backward: a chunk's gate and up are loaded one chunk ahead.  (The activation is
// chosen outside the loops over values, and nothing in them is left out but loads and
// stores: 8191 x 6144 x 4096 212 -> 160 us.  Of these, with max(x, 0) for the activation
// 158, without the loads 148, without the stores 164 of 167 at that step; the plain
// product 116.  Eight warps with one operand stage less take 164, and 669 instead of 648
// where reading w bounds the call; loads two chunks ahead 181.)
__device__ __forceinline__ void gated_backward_epilogue(const Fp8Args& p, const Epilogue& e) {
  using L = Layout<kGatedBackward>;
  static_assert(L::kOutBufs * L::kOutBuf >= 32 * 32 * 4, "one FP32 chunk per warp");
  float* buf = reinterpret_cast<float*>(e.out + e.quad * L::kOutBufs * L::kOutBuf);
  int acc = 0;
  uint32_t phase = 0;
  Tile o;
  for (uint32_t t = e.pair; decode<kGatedBackward>(p, e.first, e.start, t, o); t += e.npairs) {
    const int n = o.n0 + static_cast<int>(e.rank) * kHalfM + e.quad * 32 + (e.lane & 3) * 8;
    const int chunks = (o.cols + 31) / 32;
    const int64_t base = static_cast<int64_t>(o.c0) * p.n + n;
    uint4 gate[4] = {}, up[4] = {};
    const auto load = [&](int cb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = cb * 32 + i * 8 + (e.lane >> 2);
        if (tok < o.cols && n < p.n) {
          const int64_t at = base + static_cast<int64_t>(tok) * p.n;
          gate[i] = *reinterpret_cast<const uint4*>(p.gate + at);
          up[i] = *reinterpret_cast<const uint4*>(p.up + at);
        }
      }
    };
    load(0);
    if (!warp_wait(&e.full[acc], phase, e.abort_flag)) {
      e.give_up(p.err);
      break;
    }
    ptx::tc_fence_after();
    const uint32_t taddr = e.tmem + (static_cast<uint32_t>(e.quad * 32) << 16) +
                           static_cast<uint32_t>(acc * L::kAccCols);
    for (int cb = 0; cb < chunks; ++cb) {
      uint32_t v[32];
      __syncwarp();                                 // the last chunk has been read
      ptx::tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(cb * 32), v);
      ptx::tmem_ld_wait();
      if (cb == chunks - 1) e.hand_back(acc);
      put_chunk(buf, e.lane, v);
      uint4 g4[4], u4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g4[i] = gate[i];
        u4[i] = up[i];
      }
      if (cb + 1 < chunks) load(cb + 1);
      __syncwarp();
      with_activation(p.activation, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tt = i * 8 + (e.lane >> 2), tok = cb * 32 + tt;
          Pair d[4], g[4], u[4], dg[4], du[4];
          get_columns(buf, tt, (e.lane & 3) * 8, d);
          unpack_bf16(g4[i], g);
          unpack_bf16(u4[i], u);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            Pair slope;
            const Pair f = activate<kind.value, true>(g[q], &slope);
            dg[q] = mul2(mul2(d[q], u[q]), slope);
            du[q] = mul2(d[q], f);
            g[q] = mul2(f, u[q]);
          }
          if (tok < o.cols && n < p.n) {
            const int64_t to = base + static_cast<int64_t>(tok) * p.n;
            *reinterpret_cast<uint4*>(p.grad_gate + to) = pack_bf16(dg);
            *reinterpret_cast<uint4*>(p.grad_up + to) = pack_bf16(du);
            if (p.y != nullptr) *reinterpret_cast<uint4*>(p.y + to) = pack_bf16(g);
          }
        }
      });
    }
    acc ^= 1;
    if (acc == 0) phase ^= 1u;
  }
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<MODE>::kThreads, 1)
    fp8_product_kernel(const __grid_constant__ Maps<MODE> maps, const Fp8Args p) {
  using L = Layout<MODE>;
  constexpr bool GRAD = MODE == kWgrad;
  constexpr int kHalves = MODE == kSum ? 2 : 1;   // products summed in the accumulator
  constexpr int kStages = L::kMaxStages, kSets = L::kSets;
  const int stage_bytes = MODE == kGated ? p.stage_bytes : L::kStageBytes;
  const int stages = p.stages;
  constexpr int kEpiWarps = L::kEpiWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  int32_t* first = reinterpret_cast<int32_t*>(smem + L::kTableAt);
  int32_t* start = reinterpret_cast<int32_t*>(smem + L::kTableAt + L::kTableBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarAt);
  uint64_t* empty = full + kStages;
  uint64_t* set_full = empty + kStages;
  uint64_t* set_empty = set_full + kSets;
  uint64_t* tmem_full = set_empty + kSets;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* drain = tmem_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int64_t* warp_total = reinterpret_cast<int64_t*>(tmem_holder + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSets; ++s) {
      ptx::mbar_init(&set_full[s], 2);            // both CTAs' scales
      ptx::mbar_init(&set_empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tmem_full[a], 1);
      ptx::mbar_init(&tmem_empty[a], 2 * kEpiWarps);
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&maps.a);
    if (GRAD) ptx::tma_prefetch_desc(&maps.out);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_holder, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_dep_wait();
  grid_dep_launch();
  scan_experts<MODE>(p, first, start, warp_total);
  __syncthreads();

  if (warp == 0) {
    // ------------------------------------------------------------ producers
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      Tile o;
      for (uint32_t t = pair; ok && decode<MODE>(p, first, start, t, o); t += npairs) {
        const int half = o.width / 2;
        const int box = GRAD ? 0 : o.width / kWidthUnit - 1;
        const uint32_t b_bytes = static_cast<uint32_t>(half * kBK);
        const uint32_t a_bytes = MODE == kGated ? static_cast<uint32_t>(p.tile * kBK) : kABytes;
        const int row_a = o.n0 + static_cast<int>(rank) * (tile_rows<MODE>(p) / 2);
        const int row_b = o.c0 + static_cast<int>(rank) * half;
        for (int step = 0; step < kHalves * o.nkb; ++step) {
          const bool second = kHalves > 1 && step >= o.nkb;
          const int kb = second ? step - o.nkb : step;
          if (!ptx::mbar_wait_cluster(&empty[stage], phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t full_leader = ptx::mapa_shared(ptx::smem_addr(&full[stage]), 0);
          if (leader) ptx::mbar_arrive_expect_tx(&full[stage], 2u * (a_bytes + b_bytes));
          uint8_t* sa = smem + stage * stage_bytes;
          ptx::tma_load_3d_pair(sa, second ? &maps.out : &maps.a, full_leader, (o.kb0 + kb) * kBK,
                                row_a, GRAD ? 0 : o.expert);
          if (MODE == kGated)
            ptx::tma_load_3d_pair(sa + kABytes / 2, &maps.out, full_leader, kb * kBK, row_a, o.expert);
          const CUtensorMap* map_b = &maps.b[box];
          if constexpr (MODE == kSum) {
            if (second) map_b = &maps.b2[box];
          }
          ptx::tma_load_3d_pair(sa + kABytes, map_b, full_leader, (o.kb0 + kb) * kBK, row_b, 0);
          ++issued;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.err, kDevErrTimeout);
      }
      const int pending = issued < stages ? issued : stages;
      for (int j = 0; j < pending; ++j) {
        if (stage == 0) {
          stage = stages;
          phase ^= 1u;
        }
        --stage;
        ptx::mbar_wait_cluster(&empty[stage], phase, nullptr);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // The whole warp walks the loop and one elected lane issues: addresses and
    // descriptors are then the same in all lanes and stay in uniform
    // registers, where these instructions want them.
    if (leader) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      int set = 0;
      uint32_t set_phase = 0;
      bool ok = true;
      const uint64_t a_desc0 = ptx::smem_desc_sw128(ptx::smem_addr(smem), 16, 1024);
      const uint64_t s_desc0 = ptx::smem_desc_scales(ptx::smem_addr(smem + L::kScaleAt));
      Tile o;
      for (uint32_t t = pair; ok && decode<MODE>(p, first, start, t, o); t += npairs) {
        if (o.nkb == 0) continue;
        if (!warp_wait(&tmem_empty[acc], acc_phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * L::kAccCols);
        const uint32_t idesc0 = ptx::idesc_mxf8(kTileM, o.width);
        const bool wide = o.width > 128;
        int half = 0;
        for (int kb0 = 0; ok && kb0 < o.nkb;) {
          if (!warp_wait(&set_full[set], set_phase, abort_flag)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          // Two sets of scale cells in TMEM in turn.
          const uint32_t sa_tmem = tmem_base + kTmemScales + (set & 1) * 16, sb_tmem = sa_tmem + 4;
          const uint64_t s_desc = s_desc0 + static_cast<uint32_t>(set * (kScaleBytes >> 4));
          if (ptx::elect_one()) {
            ptx::tc_copy_scales_pair(sa_tmem, s_desc);
            ptx::tc_copy_scales_pair(sb_tmem, s_desc + (512 >> 4));
            if (wide) ptx::tc_copy_scales_pair(sb_tmem + 4, s_desc + (1024 >> 4));
          }
          __syncwarp();
#pragma unroll
          for (int b = 0; b < kSetBlocks; ++b) {
            if (kb0 + b >= o.nkb) break;
            if (!warp_wait(&full[stage], phase, abort_flag)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint32_t idesc = ptx::idesc_mxf8_byte(idesc0, b);
            const uint64_t a_desc = a_desc0 + static_cast<uint32_t>(stage * (stage_bytes >> 4));
            const uint64_t b_desc = a_desc + (kABytes >> 4);
            const int steps = kb0 + b == o.nkb - 1 ? o.last : kBK / 32;
            if (ptx::elect_one()) {
#pragma unroll
              for (int k = 0; k < kBK / 32; ++k)
                if (k < steps)
                  ptx::tc_mma_mxf8_pair(d_tmem, a_desc + k * 2, b_desc + k * 2, idesc, sa_tmem, sb_tmem,
                                        (half | kb0 | b | k) != 0 ? 1u : 0u);
              ptx::tc_commit_pair_multicast(&empty[stage], 0x3);
            }
            __syncwarp();
            if (++stage == stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (ptx::elect_one()) ptx::tc_commit_pair_multicast(&set_empty[set], 0x3);
          __syncwarp();
          if (++set == kSets) {
            set = 0;
            set_phase ^= 1u;
          }
          kb0 += kSetBlocks;
          if (kHalves > 1 && half == 0 && kb0 >= o.nkb) {
            half = 1;
            kb0 = 0;
          }
        }
        if (!ok) break;
        if (ptx::elect_one()) ptx::tc_commit_pair_multicast(&tmem_full[acc], 0x3);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        atomicOr(p.err, kDevErrTimeout);
      }
      if (ptx::elect_one()) ptx::tc_commit_pair(drain);
      __syncwarp();
      ptx::mbar_wait(drain, 0, nullptr);
    }
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    if constexpr (MODE == kGated || MODE == kGatedBackward) {
      const Epilogue e{first, start, smem + L::kOutAt, tmem_base, tmem_full, tmem_empty, abort_flag,
                       rank, pair, npairs, warp & 3, lane};
      if constexpr (MODE == kGated)
        gated_epilogue(p, e);
      else
        gated_backward_epilogue(p, e);
    } else {
      const int quad = warp & 3;
      int acc = 0;
      uint32_t acc_phase = 0;
      const uint32_t empty_leader0 = ptx::mapa_shared(ptx::smem_addr(&tmem_empty[0]), 0);
      const uint32_t empty_leader1 = ptx::mapa_shared(ptx::smem_addr(&tmem_empty[1]), 0);
      uint8_t* stage_out = smem + L::kOutAt + (warp - 2) * L::kOutBufs * L::kOutBuf;
      int issued = 0;
      // dw is far larger than L2: written lines leave it in the order they came
      // (64 experts of 2048 x 8704: 775 -> 723 us).
      const uint64_t leave_first = ptx::l2_evict_first();
      Tile o;
      for (uint32_t t = pair; decode<MODE>(p, first, start, t, o); t += npairs) {
        const int row0 = o.n0 + static_cast<int>(rank) * kHalfM + quad * 32;
        const bool empty_sum = o.nkb == 0;
        if (empty_sum && p.accumulate) continue;
        if (!empty_sum) {
          if (!warp_wait(&tmem_full[acc], acc_phase, abort_flag)) {
            if (lane == 0) {
              *abort_flag = 1;
              atomicOr(p.err, kDevErrTimeout);
            }
            break;
          }
          ptx::tc_fence_after();
        }
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                               static_cast<uint32_t>(acc * L::kAccCols);
        for (int cb = 0; cb * 32 < o.cols; ++cb) {
          uint32_t v[32];
          __syncwarp();
          if (!empty_sum) {
            ptx::tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(cb * 32), v);
            ptx::tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          }
          if (GRAD && row0 >= p.n) continue;
          uint8_t* buf = stage_out + (issued % L::kOutBufs) * L::kOutBuf;
          ++issued;
          if (GRAD) {
            // 32 rows x 128 bytes, 16-byte chunk q of row r at q ^ (r & 7): the
            // output map's 128-byte swizzle.  A buffer is free once the store
            // issued from it has read it.
            if (lane == 0) ptx::bulk_wait_read<L::kOutBufs - 1>();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                  make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (p.accumulate)
                ptx::tma_reduce_add_3d(&maps.out, buf, o.c0 + cb * 32, row0, o.expert);
              else
                ptx::tma_store_3d_hint(&maps.out, buf, o.c0 + cb * 32, row0, o.expert, leave_first);
              ptx::bulk_commit();
            }
          } else {
            // A lane holds one output column of 32 tokens.  Two tokens' values
            // rounded to BF16 make a word (half the stores to shared memory, which
            // bound tiles with few K blocks); a lane then takes the words of eight
            // columns, and halves of them are 16 bytes of either token.  Odd pairs'
            // words are stored four places round, so that both halves' reads hit
            // all banks.
            uint32_t* words = reinterpret_cast<uint32_t*>(buf);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const __nv_bfloat162 two =
                  __floats2bfloat162_rn(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
              words[q * 32 + (lane ^ ((q & 1) << 2))] = *reinterpret_cast<const uint32_t*>(&two);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int pr = i * 8 + (lane >> 2), g = lane & 3;
              const int at = pr * 32 + ((g * 8) ^ ((pr & 1) << 2));
              const uint4 lo = *reinterpret_cast<const uint4*>(words + at);
              const uint4 hi = *reinterpret_cast<const uint4*>(words + (at ^ 4));
              const int tok = cb * 32 + 2 * pr, n = row0 + g * 8;
              __nv_bfloat16* to = p.y + static_cast<int64_t>(o.c0 + tok) * p.n + n;
              if (tok < o.cols && n < p.n)
                *reinterpret_cast<uint4*>(to) =
                    make_uint4(__byte_perm(lo.x, lo.y, 0x5410), __byte_perm(lo.z, lo.w, 0x5410),
                               __byte_perm(hi.x, hi.y, 0x5410), __byte_perm(hi.z, hi.w, 0x5410));
              if (tok + 1 < o.cols && n < p.n)
                *reinterpret_cast<uint4*>(to + p.n) =
                    make_uint4(__byte_perm(lo.x, lo.y, 0x7632), __byte_perm(lo.z, lo.w, 0x7632),
                               __byte_perm(hi.x, hi.y, 0x7632), __byte_perm(hi.z, hi.w, 0x7632));
            }
          }
        }
        if (!empty_sum) {
          // Every value has been read into registers and staged.
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster_relaxed(acc ? empty_leader1 : empty_leader0);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      if (GRAD && lane == 0) ptx::bulk_wait_all();
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ scales (both CTAs)
    // Warp `which` fills the sets which, which + scale_warps, ...; a set's loads
    // are in flight while it waits for its place.  They follow the arrival for
    // the set before: a release waits for its thread's loads too.  A set takes a
    // warp some 3000 cycles (loads, proxy fence, release): four warps keep up with
    // tiles of a few K blocks (25599 x 2768 x 576: 83 us with two, 60 with four).
    const int which = warp - 2 - kEpiWarps;
    SetCursor at{};
    at.begin<MODE>(p, first, start, pair);
    at.settle<MODE>(p, first, start, npairs);
    at.advance<MODE>(p, first, start, npairs, which);
    if (which >= p.scale_warps) at.live = false;  // not in use
    int set = which;
    uint32_t set_phase = 0;
    bool ok = true;
    while (at.live) {
      uint32_t cells[kCells];
      load_set<MODE>(p, at, rank, lane, cells);
      at.advance<MODE>(p, first, start, npairs, p.scale_warps);
      if (!warp_wait(&set_empty[set], set_phase ^ 1u, abort_flag)) {
        ok = false;
        break;
      }
      // Lane l's 16 bytes hold the cells of rows l, l + 32, l + 64, l + 96.
      uint4* to = reinterpret_cast<uint4*>(smem + L::kScaleAt + set * kScaleBytes);
      to[lane] = make_uint4(cells[0], cells[1], cells[2], cells[3]);
      to[32 + lane] = make_uint4(cells[4], cells[5], cells[6], cells[7]);
      to[64 + lane] = make_uint4(cells[8], cells[9], cells[10], 0u);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          ptx::mbar_arrive(&set_full[set]);
        else
          ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(&set_full[set]), 0));
      }
      set += p.scale_warps;
      if (set >= kSets) {
        set -= kSets;
        set_phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, kDevErrTimeout);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The installed driver's cuTensorMapEncodeTiled (NULL: unavailable).
inline EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeFn>(ptr);
  }();
  return fn;
}

// (cols, rows, count) of bytes or FP32 values, 128-byte swizzle, zero fill.
inline bool encode(CUtensorMap* map, bool fp32, const void* ptr, int64_t cols, int64_t rows, int64_t count,
            int box_cols, int box_rows) {
  const EncodeFn enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t el = fp32 ? 4 : 1;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(count)};
  const cuuint64_t strides[2] = {dims[0] * el, dims[0] * dims[1] * el};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1u};
  const cuuint32_t step[3] = {1u, 1u, 1u};
  return enc(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
             const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t setup(int num_sms, int* pairs) {
  const cudaError_t e = cudaFuncSetAttribute(
      fp8_product_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<MODE>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(Layout<MODE>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<MODE>::kSmem;
  return resident_pairs(
      [&](int* n) { return cudaOccupancyMaxActiveClusters(n, fp8_product_kernel<MODE>, &cfg); },
      num_sms, pairs);
}

template <int MODE>
cudaError_t launch(const Maps<MODE>& maps, const Fp8Args& p, int64_t max_tiles, int64_t pairs,
                   cudaStream_t s) {
  if (pairs > max_tiles) pairs = max_tiles;
  if (pairs < 1) pairs = 1;
  if (max_tiles + 2 * pairs >= INT32_MAX) return cudaErrorInvalidValue;   // tile numbers are 32 bits
  return launch_pdl(fp8_product_kernel<MODE>, dim3(static_cast<unsigned>(2 * pairs)),
                    dim3(Layout<MODE>::kThreads),
                    Layout<MODE>::kSmem, s, maps, p);
}

}  // namespace fp8
}  // namespace muon
