// k_fp8_gemm.cu -- the experts' products on FP8 operands with a power-of-two
// scale per 128 values, on CTA pairs (tcgen05 cta_group::2, block-scaled MMA).
//
//   rows   y[r] = sum_b 2^(sx[r,b] + sw[e,n/128,b]) sum_{k in block b} x[r,k] w[e,n,k]
//          for the rows r of expert e (forward; with the transposed weights the
//          gradient of the input)
//   wgrad  dw[e] = sum over the expert's blocks of 128 rows of dY^T X, each
//          operand scaled per (128 rows, column)
//
// Both have the weights' output rows on the accumulator's lanes (256 per pair
// tile, 128 per CTA) and, on its columns, an expert's tokens (rows) or the
// weights' input columns (wgrad).  Tokens are the ragged side: an MMA may have
// any multiple of 32 columns, so an expert's tokens are cut into
// ceil(M / 224) tiles of equal width instead of being padded to 128.  224 is
// the widest that leaves room in TMEM for the scales beside two accumulators
// (2 x 224 + 32 <= 512 columns).
//
// The tensor cores multiply by the scales: each 128-wide K block is four MMAs
// (K = 32) that read one scale byte per row of A and of B from TMEM, where a
// 32-bit cell holds the bytes of four K blocks.  Up to four warps per CTA gather
// four blocks' bytes of the tile's rows at a time (a set), write them to a ring in
// shared memory apart from the operands', and the MMA thread copies a set to TMEM
// (tcgen05.cp) ahead of its MMAs.  Sets are counted from the tile's first K block,
// so rows need no alignment.
//
// A persistent pair walks the tiles.  Warp 0: TMA producer.  Warp 1: TMEM and,
// in the even CTA, the MMAs.  Then the epilogue's warps, overlapped with
// the next tile through the second accumulator, and the scales'.  The experts' rows
// are read from `offsets` on the device: every block sums the experts' tile
// counts before its first tile, so a call needs no host copy of the routing.
//
// Bound and measured (GB300).  Rows with few tokens per expert: reading w, 512
// experts of 1536 x 4096 with 57344 rows 531-550 us (3.63 GB, 6.6-6.8 TB/s).
// Dense: the tensor pipe at the power cap, 16381 x 6144 x 4096 280 us in a stream
// of calls (2.9 PFLOP/s), 240 us by itself (3.4 PFLOP/s, pipe 89% active).  One
// token through 7 experts: latency, 15.1-15.5 us.  Weight gradient with few tokens
// per expert: writing dw, 64 experts of 2048 x 8704 725-765 us (4.66 GB, 6.1-6.4
// TB/s), added to what is there 1840 us (floor 1356).  With one expert the tiles
// are few: 16384 rows into 6144 x 4096 261 us (floor 217), but into 1024 x 1024
// 50 us (floor 9) and 4096 x 272 54 us (floor 11).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_ptx.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "moe.h"

namespace muon {
namespace {

constexpr int kTileM = 256;                       // pair tile: output rows of w / dw
constexpr int kHalfM = 128;
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

template <bool GRAD>
struct Layout {
  static constexpr int kEpiWarps = 4;                         // one per 32 lanes (eight: no faster)
  static constexpr int kScaleWarps = 4;                       // at most
  static constexpr int kSets = 8;                             // sets of scales in the ring
  static constexpr int kThreads = 32 * (2 + kEpiWarps + kScaleWarps);
  static constexpr int kAccCols = GRAD ? kGradN : kMaxTokens;
  static constexpr int kStages = GRAD ? 5 : 6;                // operand stages, at most
  static constexpr int kOutBufs = 2;                          // per epilogue warp
  static constexpr int kBBytes = (kAccCols / 2) * kBK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kOutBuf = GRAD ? 4096 : 2048;          // one 32 x 32 chunk
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
  const int32_t* offsets;
  int32_t experts;
  int32_t n;            // rows of w / dw
  int32_t k;            // rows: contraction; wgrad: columns of dw
  int64_t rows;         // rows: rows of x and y; wgrad: columns of yt and xt
  int32_t n_blocks, k_blocks;
  int32_t tiles_m, tiles_n;
  __nv_bfloat16* y;
  int32_t stages;       // operand stages in use
  int32_t scale_warps;  // scale warps in use (a divisor of kSets)
  int32_t accumulate;
  int* err;
};

struct Maps {
  CUtensorMap a;
  CUtensorMap b[kMaps];
  CUtensorMap out;
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

// first[e]: token tiles (rows) or row blocks (wgrad) before expert e;
// start[e]: its first row (rows) or how many rows it has (wgrad).
template <bool GRAD>
__device__ __forceinline__ bool decode(const Fp8Args& p, const int32_t* first, const int32_t* start,
                                       uint32_t t, Tile& o) {
  const uint32_t tiles_m = p.tiles_m;
  if (GRAD) {
    const uint32_t per = tiles_m * p.tiles_n;
    o.expert = static_cast<int>(t / per);
    if (o.expert >= p.experts) return false;
    const uint32_t l = t - o.expert * per;
    // Along a row of tiles first: the pairs running at one time then write
    // whole rows of dw.
    const uint32_t tm = l / p.tiles_n;
    o.n0 = static_cast<int>(tm) * kTileM;
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
  o.n0 = static_cast<int>(tm) * kTileM;
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
template <bool GRAD>
__device__ __forceinline__ void scan_experts(const Fp8Args& p, int32_t* first, int32_t* start,
                                             int64_t* warp_total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kPer = kMoeMaxExperts / Layout<GRAD>::kThreads + 1;   // and the end of the last
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

// Walks the sets of scales of a pair's tiles.
struct SetCursor {
  uint32_t t;
  Tile o;
  int kb;               // first K block of the set
  bool live;

  template <bool GRAD>
  __device__ __forceinline__ void begin(const Fp8Args& p, const int32_t* first, const int32_t* start,
                                        uint32_t t0) {
    t = t0;
    kb = 0;
    live = decode<GRAD>(p, first, start, t, o);
  }
  // Leaves a tile without K blocks at once.
  template <bool GRAD>
  __device__ __forceinline__ void settle(const Fp8Args& p, const int32_t* first,
                                         const int32_t* start, int step) {
    while (live && kb >= o.nkb) {
      t += step;
      kb = 0;
      live = decode<GRAD>(p, first, start, t, o);
    }
  }
  // `sets` sets further.
  template <bool GRAD>
  __device__ __forceinline__ void advance(const Fp8Args& p, const int32_t* first,
                                          const int32_t* start, int step, int sets) {
    for (int i = 0; i < sets && live; ++i) {
      kb += kSetBlocks;
      settle<GRAD>(p, first, start, step);
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

template <bool GRAD>
__device__ __forceinline__ void load_set(const Fp8Args& p, const SetCursor& s, uint32_t rank,
                                         int lane, uint32_t (&cells)[kCells]) {
  const Tile& o = s.o;
  const int row_a = o.n0 + static_cast<int>(rank) * kHalfM;
  const int n = min(kSetBlocks, o.nkb - s.kb);
  constexpr int kB = kCells - 4;
  uint32_t off[kB];
  if (GRAD) {
    const int64_t kb = o.kb0 + s.kb;
    uint32_t off_a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) off_a[i] = min(row_a + i * 32 + lane, p.n - 1);
#pragma unroll
    for (int i = 0; i < kB; ++i) off[i] = min(o.c0 + i * 32 + lane, p.k - 1);
    load_cells<4>(p.a_scales + kb * p.n, p.n, n, off_a, cells);
    load_cells<kB>(p.b_scales + kb * p.k, p.k, n, off, cells + 4);
  } else {
    const uint8_t* a = p.a_scales + s.kb + (static_cast<int64_t>(o.expert) * p.n_blocks +
                                            min(row_a / kBK, p.n_blocks - 1)) * p.k_blocks;
    const uint8_t* b = p.b_scales + s.kb + static_cast<int64_t>(o.c0) * p.k_blocks;
#pragma unroll
    for (int i = 0; i < kB; ++i) off[i] = min(i * 32 + lane, o.cols - 1) * p.k_blocks;
    // Rows of a multiple of four blocks start on a word (the buffers are
    // 16-byte aligned): one load per row.
    if (p.k_blocks % kSetBlocks == 0) {
      cells[0] = __ldg(reinterpret_cast<const uint32_t*>(a));
#pragma unroll
      for (int i = 0; i < kB; ++i) cells[4 + i] = __ldg(reinterpret_cast<const uint32_t*>(b + off[i]));
    } else {
      const uint32_t zero[1] = {0u};
      load_cells<1>(a, 1, n, zero, cells);
      load_cells<kB>(b, 1, n, off, cells + 4);
    }
#pragma unroll
    for (int i = 1; i < 4; ++i) cells[i] = cells[0];
  }
}

template <bool GRAD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<GRAD>::kThreads, 1)
    fp8_product_kernel(const __grid_constant__ Maps maps, const Fp8Args p) {
  using L = Layout<GRAD>;
  constexpr int kStages = L::kStages, kSets = L::kSets;
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
  scan_experts<GRAD>(p, first, start, warp_total);
  __syncthreads();

  if (warp == 0) {
    // ------------------------------------------------------------ producers
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      Tile o;
      for (uint32_t t = pair; ok && decode<GRAD>(p, first, start, t, o); t += npairs) {
        const int half = o.width / 2;
        const int box = GRAD ? 0 : o.width / kWidthUnit - 1;
        const uint32_t b_bytes = static_cast<uint32_t>(half * kBK);
        const int row_a = o.n0 + static_cast<int>(rank) * kHalfM;
        const int row_b = o.c0 + static_cast<int>(rank) * half;
        for (int kb = 0; kb < o.nkb; ++kb) {
          if (!ptx::mbar_wait_cluster(&empty[stage], phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t full_leader = ptx::mapa_shared(ptx::smem_addr(&full[stage]), 0);
          if (leader) ptx::mbar_arrive_expect_tx(&full[stage], 2u * (kABytes + b_bytes));
          uint8_t* sa = smem + stage * L::kStageBytes;
          ptx::tma_load_3d_pair(sa, &maps.a, full_leader, (o.kb0 + kb) * kBK, row_a,
                                GRAD ? 0 : o.expert);
          ptx::tma_load_3d_pair(sa + kABytes, &maps.b[box], full_leader, (o.kb0 + kb) * kBK, row_b,
                                0);
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
      for (uint32_t t = pair; ok && decode<GRAD>(p, first, start, t, o); t += npairs) {
        if (o.nkb == 0) continue;
        if (!warp_wait(&tmem_empty[acc], acc_phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * L::kAccCols);
        const uint32_t idesc0 = ptx::idesc_mxf8(kTileM, o.width);
        const bool wide = o.width > 128;
        for (int kb0 = 0; ok && kb0 < o.nkb; kb0 += kSetBlocks) {
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
            const uint64_t a_desc = a_desc0 + static_cast<uint32_t>(stage * (L::kStageBytes >> 4));
            const uint64_t b_desc = a_desc + (kABytes >> 4);
            const int steps = kb0 + b == o.nkb - 1 ? o.last : kBK / 32;
            if (ptx::elect_one()) {
#pragma unroll
              for (int k = 0; k < kBK / 32; ++k)
                if (k < steps)
                  ptx::tc_mma_mxf8_pair(d_tmem, a_desc + k * 2, b_desc + k * 2, idesc, sa_tmem, sb_tmem,
                                        (kb0 | b | k) != 0 ? 1u : 0u);
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
    for (uint32_t t = pair; decode<GRAD>(p, first, start, t, o); t += npairs) {
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
  } else {
    // ------------------------------------------------------------ scales (both CTAs)
    // Warp `which` fills the sets which, which + scale_warps, ...; a set's loads
    // are in flight while it waits for its place.  They follow the arrival for
    // the set before: a release waits for its thread's loads too.  A set takes a
    // warp some 3000 cycles (loads, proxy fence, release): four warps keep up with
    // tiles of a few K blocks (25599 x 2768 x 576: 83 us with two, 60 with four).
    const int which = warp - 2 - kEpiWarps;
    SetCursor at{};
    at.begin<GRAD>(p, first, start, pair);
    at.settle<GRAD>(p, first, start, npairs);
    at.advance<GRAD>(p, first, start, npairs, which);
    if (which >= p.scale_warps) at.live = false;  // not in use
    int set = which;
    uint32_t set_phase = 0;
    bool ok = true;
    while (at.live) {
      uint32_t cells[kCells];
      load_set<GRAD>(p, at, rank, lane, cells);
      at.advance<GRAD>(p, first, start, npairs, p.scale_warps);
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
EncodeFn encoder() {
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
bool encode(CUtensorMap* map, bool fp32, const void* ptr, int64_t cols, int64_t rows, int64_t count,
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

template <bool GRAD>
cudaError_t setup(int num_sms, int* pairs) {
  const cudaError_t e = cudaFuncSetAttribute(
      fp8_product_kernel<GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<GRAD>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(Layout<GRAD>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<GRAD>::kSmem;
  return resident_pairs(
      [&](int* n) { return cudaOccupancyMaxActiveClusters(n, fp8_product_kernel<GRAD>, &cfg); },
      num_sms, pairs);
}

template <bool GRAD>
cudaError_t launch(const Maps& maps, const Fp8Args& p, int64_t max_tiles, int64_t pairs,
                   cudaStream_t s) {
  if (pairs > max_tiles) pairs = max_tiles;
  if (pairs < 1) pairs = 1;
  if (max_tiles + 2 * pairs >= INT32_MAX) return cudaErrorInvalidValue;   // tile numbers are 32 bits
  return launch_pdl(fp8_product_kernel<GRAD>, dim3(static_cast<unsigned>(2 * pairs)),
                    dim3(Layout<GRAD>::kThreads),
                    Layout<GRAD>::kSmem, s, maps, p);
}

}  // namespace

cudaError_t fp8_gemm_init(int num_sms, Fp8Pairs* pairs) {
  const cudaError_t e = setup<false>(num_sms, &pairs->matmul);
  return e != cudaSuccess ? e : setup<true>(num_sms, &pairs->wgrad);
}

cudaError_t launch_fp8_grouped_matmul(const uint8_t* x, const uint8_t* x_scales, const uint8_t* w,
                                      const uint8_t* w_scales, const int32_t* offsets, int experts,
                                      int64_t rows, int n, int k, uint16_t* y, int* err, int pairs,
                                      cudaStream_t s) {
  Maps maps;
  bool ok = encode(&maps.a, false, w, k, n, experts, kBK, kHalfM);
  for (int i = 0; i < kMaps; ++i)
    ok = ok && encode(&maps.b[i], false, x, k, rows, 1, kBK, (i + 1) * (kWidthUnit / 2));
  if (!ok) return cudaErrorInvalidValue;
  maps.out = maps.a;
  Fp8Args p{};
  p.a_scales = w_scales;
  p.b_scales = x_scales;
  p.offsets = offsets;
  p.experts = experts;
  p.n = n;
  p.k = k;
  p.rows = rows;
  p.n_blocks = (n + kBK - 1) / kBK;
  p.k_blocks = (k + kBK - 1) / kBK;
  p.tiles_m = (n + kTileM - 1) / kTileM;
  p.stages = Layout<false>::kStages;
  p.scale_warps = Layout<false>::kScaleWarps;
  p.y = reinterpret_cast<__nv_bfloat16*>(y);
  p.err = err;
  const int64_t token_tiles = (rows < experts ? rows : experts) + rows / kMaxTokens;
  return launch<false>(maps, p, token_tiles * p.tiles_m, pairs, s);
}

cudaError_t launch_fp8_grouped_wgrad(const uint8_t* yt, const uint8_t* yt_scales,
                                     const uint8_t* xt, const uint8_t* xt_scales,
                                     const int32_t* offsets, int experts, int64_t cap, int n, int k,
                                     float* dw, bool accumulate, int* err, int pairs,
                                     cudaStream_t s) {
  Maps maps;
  bool ok = encode(&maps.out, true, dw, k, n, experts, 32, 32);
  if (cap > 0) {
    ok = ok && encode(&maps.a, false, yt, cap, n, 1, kBK, kHalfM);
    ok = ok && encode(&maps.b[0], false, xt, cap, k, 1, kBK, kGradN / 2);
  } else {
    maps.a = maps.b[0] = maps.out;                // no K block: nothing is loaded
  }
  if (!ok) return cudaErrorInvalidValue;
  for (int i = 1; i < kMaps; ++i) maps.b[i] = maps.b[0];
  Fp8Args p{};
  p.a_scales = yt_scales;
  p.b_scales = xt_scales;
  p.offsets = offsets;
  p.experts = experts;
  p.n = n;
  p.k = k;
  p.rows = cap;
  p.tiles_m = (n + kTileM - 1) / kTileM;
  p.tiles_n = (k + kGradN - 1) / kGradN;
  // Few K blocks per expert: writing dw bounds the call, and pairs that load no
  // further than the next tile stay together, so that neighbouring tiles' rows
  // leave L2 as whole runs.  Measured with 2 stages and scale warps / 5 and 4, by
  // blocks of capacity per expert (us):
  //                        1.5         2.5         3.0         3.5         5.0
  //   64 x 2048 x 8704   810/822     740/894     806/918     890/924    1135/904
  //   64 x 1536 x 4096   294/298     287/324     326/329     355/337     449/316
  //   512 x 1536 x 4096 2471/2544   2205/2827   2492/2931   2851/3041   3532/3090
  //   256 x 256 x 1024    64/64       74/74       85/76       95/81      111/89
  //   64 x 512 x 512      23/25       31/27       36/31       36/29       40/33
  // The two cross between 2.5 and 4.5, the earlier the smaller dw is; where dw
  // fits L2 they differ by a few us.  8 x 2048 x 8704 at 32: 727/403.
  const bool few = 2 * (cap / kBK) < 5 * static_cast<int64_t>(experts);
  p.stages = few ? 2 : Layout<true>::kStages;
  p.scale_warps = few ? 2 : Layout<true>::kScaleWarps;
  p.accumulate = accumulate ? 1 : 0;
  p.err = err;
  return launch<true>(maps, p, int64_t(experts) * p.tiles_m * p.tiles_n, pairs, s);
}

}  // namespace muon
