// k_fp8_quantize.cu -- FP8 (e4m3) quantisation with one power-of-two scale
// (E8M0) per block of 128, in the three layouts the grouped products read.
//
// Of a block with largest magnitude m: e = the least integer with
// m / 2^e <= 448 (the largest e4m3 value), q = e4m3(x / 2^e) to nearest even,
// stored scale byte e + 127 (a block of zeros: 127, i.e. 1).  448 = 1.75 2^8,
// so with m = f 2^p, f in [1, 2): e = p - 8, plus 1 when f > 1.75 -- read off
// the FP32 bits, and x / 2^e is an exact multiplication: the only rounding is
// to e4m3.  The tensor cores apply such scales themselves; FP32 scales would
// need every partial sum read back and multiplied.
//   rows    1 x 128 along a row; a token's row can be written to each of its
//           experts' rows (quantised once, written k times)
//   blocks  128 x 128 of a weight matrix, as it is and transposed: the same
//           scale serves the product with W and with its transpose
//   cols    128 x 1 along the rows of one expert, written transposed: the
//           operands of the weight gradient, whose sums run over rows (an
//           expert's last block only as far as the next multiple of 32 rows)
// A NaN stays NaN, an infinity becomes the largest value; both are reported
// through the device error word.  Each value is read once and written as one
// byte (two with the transpose): rows and blocks are bound by HBM (8192 tokens x
// 4096 to 7 rows each 46.5 us, 6.5 TB/s; 48 FP32 weights of 2048 x 8704 in both
// orientations 759 us, 6.8 TB/s), cols by its two barriers per tile and its
// instructions (8191 x 4096 gathered into 512 experts 110 us, 2.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "kernels.h"
#include "launch.cuh"
#include "moe.h"

namespace muon {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr uint32_t kInfBits = 0x7f800000u;

// Exponent e of the scale of a block whose largest magnitude has these FP32
// bits (an infinity: the largest finite exponent's).  The addend carries into
// the exponent field when the fraction is above 1.75's; below 2^-127 of a scale
// there is none, and 2^-127 serves.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = static_cast<int>((bits + 0x1fffffu) >> 23) - 135;
  return bits == 0u ? 0 : max(-127, e);
}

// 2^-e as FP32, -127 <= e <= 120.
__device__ __forceinline__ float inverse_scale(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// Largest magnitude as FP32 bits; NaN payloads do not take part.
__device__ __forceinline__ uint32_t mag(float v, bool& bad) {
  const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
  if (u >= kInfBits) bad = true;
  return u > kInfBits ? 0u : u;
}

// Two values times `inv` as e4m3 bytes, saturating.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b, float inv) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
}

// Two pairs of BF16 values times two pairs of scales as four bytes: mixed-
// precision FMAs (the addend -0 keeps a zero's sign) take the halves as they
// lie.
__device__ __forceinline__ uint32_t bf16_to_e4m3x4(uint32_t u, uint32_t v, uint32_t inv_u,
                                                   uint32_t inv_v) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b, c, d, p, q;\n\t.reg .f32 f, g;\n\t"
      "mov.b32 {a, b}, %1;\n\t"
      "mov.b32 {c, d}, %3;\n\t"
      "fma.rn.f32.bf16 f, a, c, 0f80000000;\n\t"
      "fma.rn.f32.bf16 g, b, d, 0f80000000;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 p, g, f;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "mov.b32 {c, d}, %4;\n\t"
      "fma.rn.f32.bf16 f, a, c, 0f80000000;\n\t"
      "fma.rn.f32.bf16 g, b, d, 0f80000000;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 q, g, f;\n\t"
      "mov.b32 %0, {p, q};\n\t}"
      : "=r"(r)
      : "r"(u), "r"(v), "r"(inv_u), "r"(inv_v));
  return r;
}

// Largest magnitudes of BF16 pairs; a NaN carries through (its bits are above
// an infinity's).
__device__ __forceinline__ uint32_t max_mag2(uint32_t m, uint32_t u) {
  const __nv_bfloat162 v = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u)));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 2^-e as BF16 bits.
__device__ __forceinline__ uint32_t inverse_scale_bf16(int e) {
  return static_cast<uint32_t>(127 - e) << 7;
}

__device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// ------------------------------------------------------------------ rows
// Eight lanes per block of 128 values, 16 values each: a row's 16 bytes per lane
// and store.
constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(
    const uint16_t* __restrict__ x, int64_t tokens, int d, int blocks,
    const int32_t* __restrict__ pos, int k, int64_t rows, const int32_t* __restrict__ live_rows,
    uint8_t* __restrict__ q, uint8_t* __restrict__ scales, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  if (live_rows != nullptr) tokens = min(tokens, static_cast<int64_t>(*live_rows));
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) >> 3;
  const int sub = threadIdx.x & 7;
  const int64_t t = unit / blocks;
  const int b = static_cast<int>(unit - t * blocks);
  const bool live = t < tokens;
  const int c = b * kFp8Block + sub * 16;
  const bool in = live && c < d;
  uint4 u = make_uint4(0, 0, 0, 0), v = u;
  if (in) {
    const uint4* from = reinterpret_cast<const uint4*>(x + t * d + c);
    u = from[0];
    v = from[1];
  }
  const uint32_t words[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t m2 = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = max_mag2(m2, words[i]);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(kAll, m2, o));
  uint32_t m = max(m2 & 0xffff0000u, m2 << 16);
  if (__any_sync(kAll, m >= kInfBits)) {          // NaN takes no part in the magnitude
    bool bad = false;
    m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max(mag(lo(words[i]), bad), mag(hi(words[i]), bad)));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
    if (bad) atomicOr(err, kDevErrInput);
  }
  if (!live) return;
  const int e = scale_exponent(m);
  const uint32_t inv = inverse_scale_bf16(e) * 0x10001u;
  const uint4 out = make_uint4(
      bf16_to_e4m3x4(u.x, u.y, inv, inv), bf16_to_e4m3x4(u.z, u.w, inv, inv),
      bf16_to_e4m3x4(v.x, v.y, inv, inv), bf16_to_e4m3x4(v.z, v.w, inv, inv));
  if (pos == nullptr) {
    if (in) *reinterpret_cast<uint4*>(q + t * d + c) = out;
    if (sub == 0) scales[t * blocks + b] = static_cast<uint8_t>(e + 127);
    return;
  }
  for (int j = 0; j < k; ++j) {
    const int r = pos[t * k + j];
    if (r < 0 || r >= rows) {
      if (r != -1) atomicOr(err, kDevErrIndex);
      continue;
    }
    if (in) *reinterpret_cast<uint4*>(q + static_cast<int64_t>(r) * d + c) = out;
    if (sub == 0) scales[static_cast<int64_t>(r) * blocks + b] = static_cast<uint8_t>(e + 127);
  }
}

// ------------------------------------------------------------------ tiles
// A 128 x 128 tile per block of 256 threads: warp w holds rows 16 w .. 16 w +
// 15, lane l columns 4 l .. 4 l + 3.  A thread's 16 rows of one column are 16
// consecutive bytes of the transposed tile, which is put together in shared
// memory (16-byte chunks, chunk index XORed with the column's group of four so
// that both the writes and the reads hit distinct banks) and written as rows
// of up to 128 bytes.
constexpr int kTileThreads = 256;

__device__ __forceinline__ uint32_t tile_chunk(int col, int chunk) {
  return static_cast<uint32_t>(col * 128 + ((chunk ^ ((col >> 2) & 7)) << 4));
}

// words[r] holds row r's four bytes of this thread; stores its 16 x 4 piece:
// 4 x 4 byte transposes.
__device__ __forceinline__ void put_transposed(uint8_t* tile, const uint32_t (&words)[16], int warp,
                                               int lane) {
  uint32_t out[4][4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t a = words[4 * g], b = words[4 * g + 1], c = words[4 * g + 2], d = words[4 * g + 3];
    const uint32_t ab = __byte_perm(a, b, 0x5140), cd = __byte_perm(c, d, 0x5140);
    const uint32_t ef = __byte_perm(a, b, 0x7362), gh = __byte_perm(c, d, 0x7362);
    out[0][g] = __byte_perm(ab, cd, 0x5410);
    out[1][g] = __byte_perm(ab, cd, 0x7632);
    out[2][g] = __byte_perm(ef, gh, 0x5410);
    out[3][g] = __byte_perm(ef, gh, 0x7632);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(tile + tile_chunk(lane * 4 + c, warp)) =
        make_uint4(out[c][0], out[c][1], out[c][2], out[c][3]);
}

// Rows (the source's columns) of the transposed tile to dst, `width` bytes
// (a multiple of 16) each.
__device__ __forceinline__ void write_transposed(const uint8_t* tile, uint8_t* dst, int64_t pitch,
                                                 int cols, int width) {
#pragma unroll
  for (int i = 0; i < 128 * 8 / kTileThreads; ++i) {
    const int at = i * kTileThreads + threadIdx.x;
    const int col = at >> 3, chunk = at & 7;
    if (col < cols && chunk * 16 < width)
      *reinterpret_cast<uint4*>(dst + col * pitch + chunk * 16) =
          *reinterpret_cast<const uint4*>(tile + tile_chunk(col, chunk));
  }
}

__device__ __forceinline__ float4 load_weights(const void* w, int64_t at) {
  return __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(w) + at));
}

__global__ void __launch_bounds__(kTileThreads) quantize_blocks_kernel(
    const void* __restrict__ w, int n, int k, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scales, uint8_t* __restrict__ qt, uint8_t* __restrict__ scales_t,
    int* err) {
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ uint32_t warp_max[kTileThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nb = (n + kFp8Block - 1) / kFp8Block, kb = (k + kFp8Block - 1) / kFp8Block;
  const int per = nb * kb;
  const int64_t expert = blockIdx.x / per;
  const int in_expert = static_cast<int>(blockIdx.x - expert * per);
  const int bn = in_expert / kb, bk = in_expert - bn * kb;
  const int n0 = bn * kFp8Block, k0 = bk * kFp8Block;
  const int row0 = n0 + warp * 16, col = k0 + lane * 4;
  const int64_t base = expert * n * k;

  float4 v[16];
  bool bad = false;
  uint32_t m = 0u;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    v[r] = row0 + r < n && col < k ? load_weights(w, base + static_cast<int64_t>(row0 + r) * k + col)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < 16; ++r)
    m = max(max(m, max(mag(v[r].x, bad), mag(v[r].y, bad))), max(mag(v[r].z, bad), mag(v[r].w, bad)));
  m = __reduce_max_sync(kAll, m);
  if (bad) atomicOr(err, kDevErrInput);
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileThreads / 32; ++i) m = max(m, warp_max[i]);
  const int e = scale_exponent(m);
  const float inv = inverse_scale(e);
  uint32_t words[16];
#pragma unroll
  for (int r = 0; r < 16; ++r)
    words[r] = to_e4m3x2(v[r].x, v[r].y, inv) | (to_e4m3x2(v[r].z, v[r].w, inv) << 16);
  // The transpose first: with q's rows stored before the barrier the kernel took
  // 990 us instead of 757 (48 x 2048 x 8704).
  if (qt != nullptr) {
    put_transposed(tile, words, warp, lane);
    __syncthreads();
    write_transposed(tile, qt + base + static_cast<int64_t>(k0) * n + n0, n, min(kFp8Block, k - k0),
                     min(kFp8Block, n - n0));
    if (threadIdx.x == 0) scales_t[(expert * kb + bk) * nb + bn] = static_cast<uint8_t>(e + 127);
  }
  if (q != nullptr) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (row0 + r < n && col < k)
        *reinterpret_cast<uint32_t*>(q + base + static_cast<int64_t>(row0 + r) * k + col) = words[r];
    if (threadIdx.x == 0) scales[(expert * nb + bn) * kb + bk] = static_cast<uint8_t>(e + 127);
  }
}

// BF16 weights: magnitudes and scaling on pairs, as the column quantiser; three
// blocks per SM (80 registers).  With the FP32 kernel's arithmetic on converted values the
// instructions bound it: 48 x 2048 x 4096 414 us, this one 235-238 us (the
// measured copy bandwidth).
__global__ void __launch_bounds__(kTileThreads, 3) quantize_blocks_bf16_kernel(
    const uint16_t* __restrict__ w, int n, int k, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scales, uint8_t* __restrict__ qt, uint8_t* __restrict__ scales_t,
    int* err) {
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ uint32_t warp_max[kTileThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nb = (n + kFp8Block - 1) / kFp8Block, kb = (k + kFp8Block - 1) / kFp8Block;
  const int per = nb * kb;
  const int64_t expert = blockIdx.x / per;
  const int in_expert = static_cast<int>(blockIdx.x - expert * per);
  const int bn = in_expert / kb, bk = in_expert - bn * kb;
  const int n0 = bn * kFp8Block, k0 = bk * kFp8Block;
  const int row0 = n0 + warp * 16, col = k0 + lane * 4;
  const int64_t base = expert * n * k;

  uint2 v[16];
#pragma unroll
  for (int r = 0; r < 16; ++r)
    v[r] = row0 + r < n && col < k
               ? __ldcs(reinterpret_cast<const uint2*>(w + base + static_cast<int64_t>(row0 + r) * k + col))
               : make_uint2(0u, 0u);
  uint32_t m2 = 0u;
#pragma unroll
  for (int r = 0; r < 16; ++r) m2 = max_mag2(max_mag2(m2, v[r].x), v[r].y);
  uint32_t m = max(m2 & 0xffff0000u, m2 << 16);
  if (m >= kInfBits) {                            // NaN takes no part in the magnitude
    bool bad = false;
    m = 0u;
#pragma unroll
    for (int r = 0; r < 16; ++r)
      m = max(max(m, max(mag(lo(v[r].x), bad), mag(hi(v[r].x), bad))),
              max(mag(lo(v[r].y), bad), mag(hi(v[r].y), bad)));
    if (bad) atomicOr(err, kDevErrInput);
  }
  m = __reduce_max_sync(kAll, m);
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileThreads / 32; ++i) m = max(m, warp_max[i]);
  const int e = scale_exponent(m);
  const uint32_t inv = inverse_scale_bf16(e) * 0x10001u;
  uint32_t words[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) words[r] = bf16_to_e4m3x4(v[r].x, v[r].y, inv, inv);
  if (q != nullptr) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (row0 + r < n && col < k)
        *reinterpret_cast<uint32_t*>(q + base + static_cast<int64_t>(row0 + r) * k + col) = words[r];
    if (threadIdx.x == 0) scales[(expert * nb + bn) * kb + bk] = static_cast<uint8_t>(e + 127);
  }
  if (qt != nullptr) {
    put_transposed(tile, words, warp, lane);
    __syncthreads();
    write_transposed(tile, qt + base + static_cast<int64_t>(k0) * n + n0, n, min(kFp8Block, k - k0),
                     min(kFp8Block, n - n0));
    if (threadIdx.x == 0) scales_t[(expert * kb + bk) * nb + bn] = static_cast<uint8_t>(e + 127);
  }
}

// ------------------------------------------------------------------ columns
// Persistent blocks over (chunk of kStripes 128-column stripes, block of 128
// rows of one expert), all row blocks of a chunk before the next chunk's: the
// gathered rows of a chunk (tokens x 2 KB) stay in L2 while the token's other
// experts read them, and a row block looks up its rows once per chunk.  The next
// stripe's loads are in flight while a stripe is written.
// Magnitudes are compared as pairs of 16-bit integers and values scaled by
// mixed-precision FMAs that take BF16 halves in place.  Not memory holds the
// kernel but its two barriers per stripe (the largest stall, with three blocks
// per SM at 75 registers) and its instructions (issue slots 59% busy).
constexpr int kStripes = 8;
constexpr uint32_t kNoRow = 0xffffffffu;

__global__ void __launch_bounds__(kTileThreads, 3) quantize_cols_kernel(
    const uint16_t* __restrict__ x, int64_t x_rows, int d, const int32_t* __restrict__ offsets,
    int experts, const int32_t* __restrict__ slots, int top_k, int64_t rows,
    uint8_t* __restrict__ qt, int64_t cap, uint8_t* __restrict__ scales, int* err) {
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ uint2 col_max[kTileThreads / 32][32];
  __shared__ __align__(16) uint32_t row_at[kTileThreads / 32][16];   // a warp's rows
  __shared__ int32_t first[kMoeMaxExperts + 1];   // first row block of each expert
  __shared__ int64_t warp_total[kTileThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();

  // Row blocks before each expert: an exclusive scan, 5 experts per thread (the
  // end of the last among them).  64-bit sums, cut off past the buffers' end:
  // falling offsets can count rows many times.
  constexpr int kPer = kMoeMaxExperts / kTileThreads + 1;
  const int64_t room = cap / 128;
  int count[kPer];
  int64_t sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    count[i] = 0;
    if (e < experts) {
      const int a = offsets[e], b = offsets[e + 1];
      const int n = a < 0 || b < a ? 0 : b - a;
      count[i] = n / 128 + (n % 128 != 0 ? 1 : 0);
      if (n == 0 && a != b) atomicOr(err, kDevErrIndex);
    }
    sum += count[i];
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  int64_t at = incl - sum;
  for (int i = 0; i < warp; ++i) at += warp_total[i];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e <= experts) first[e] = static_cast<int32_t>(min(at, room + 1));
    at += count[i];
  }
  __syncthreads();
  int blocks = first[experts];
  if (blocks > room) {                            // the caller's buffers are too short
    if (threadIdx.x == 0) atomicOr(err, kDevErrIndex);
    blocks = static_cast<int>(room);
  }
  const int stripes = (d + 127) / 128;
  const int64_t units = static_cast<int64_t>((stripes + kStripes - 1) / kStripes) * blocks;

  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int chunk = static_cast<int>(unit / blocks);
    const int b = static_cast<int>(unit - static_cast<int64_t>(chunk) * blocks);
    // The expert of row block b: the last one that starts at or before it.
    int lo_e = 0, hi_e = experts;
    while (hi_e - lo_e > 1) {
      const int mid = (lo_e + hi_e) >> 1;
      if (first[mid] <= b) lo_e = mid; else hi_e = mid;
    }
    const int64_t row_end = offsets[lo_e + 1];
    const int64_t block0 = offsets[lo_e] + static_cast<int64_t>(b - first[lo_e]) * 128;
    const int64_t row0 = block0 + warp * 16;
    // Rows of the block that are written: to the next multiple of 32, the K
    // step of the products.  Experts with few rows are mostly padding.
    const int width = static_cast<int>(min(int64_t(128), (row_end - block0 + 31) / 32 * 32));

    // Lane r of the warp looks up row r's source.
    int src = -1;
    if (lane < 16 && row0 + lane < row_end) {
      const int64_t r = row0 + lane;
      if (r >= 0 && r < rows) {
        src = static_cast<int>(r);
        if (slots != nullptr) {
          const int slot = slots[r];
          src = slot >= 0 ? slot / top_k : -1;
        }
      }
      if (src < 0 || src >= x_rows) {
        atomicOr(err, kDevErrIndex);
        src = -1;
      }
    }
    const bool any = __any_sync(kAll, src >= 0);  // some row of this warp is there
    const int stripe0 = chunk * kStripes, stripe1 = min(stripes, stripe0 + kStripes);
    uint2 u[16];
    const bool all = __all_sync(kAll, src >= 0 || lane >= 16);
    // Row starts in units of 16 values: 32 bits reach 2^36 values.
    __syncwarp();
    if (lane < 16)
      row_at[warp][lane] =
          src >= 0 ? static_cast<uint32_t>(src) * static_cast<uint32_t>(d >> 4) : kNoRow;
    __syncwarp();
    const auto load = [&](int stripe) {
      const int col = stripe * 128 + lane * 4;
      const uint16_t* from = x + col;
      uint32_t row[16];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint4 v = *reinterpret_cast<const uint4*>(&row_at[warp][g * 4]);
        row[4 * g] = v.x; row[4 * g + 1] = v.y; row[4 * g + 2] = v.z; row[4 * g + 3] = v.w;
      }
      if (all && stripe * 128 + 128 <= d) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          u[r] = __ldg(reinterpret_cast<const uint2*>(from + static_cast<uint64_t>(row[r]) * 16));
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          u[r] = make_uint2(0u, 0u);
          if (row[r] != kNoRow && col < d)
            u[r] = __ldg(reinterpret_cast<const uint2*>(from + static_cast<uint64_t>(row[r]) * 16));
        }
      }
    };
    if (any) load(stripe0);
    for (int stripe = stripe0; stripe < stripe1; ++stripe) {
      const int c0 = stripe * 128, col = c0 + lane * 4;
      uint2 m = make_uint2(0u, 0u);
      if (any) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          m.x = max_mag2(m.x, u[r].x);
          m.y = max_mag2(m.y, u[r].y);
        }
      }
      col_max[warp][lane] = m;
      __syncthreads();
      uint32_t words[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) words[r] = 0u;
      // Warps without rows have only zeros to give (warp 0 has the scales).
      if (any || warp == 0) {
#pragma unroll
        for (int w = 0; w < kTileThreads / 32; ++w) {
          const uint2 o = col_max[w][lane];
          m.x = __vmaxu2(m.x, o.x);
          m.y = __vmaxu2(m.y, o.y);
        }
        uint32_t top[4] = {m.x << 16, m.x & 0xffff0000u, m.y << 16, m.y & 0xffff0000u};
        if (max(max(top[0], top[1]), max(top[2], top[3])) >= kInfBits) {
          atomicOr(err, kDevErrInput);
          // NaN takes no part in the magnitude: this warp's columns again, over
          // all rows of the block.
          for (int c = 0; c < 4; ++c) {
            if (top[c] <= kInfBits) continue;
            top[c] = 0u;
            const int64_t r_begin = row0 - warp * 16, r_end = min(row_end, r_begin + 128);
            for (int64_t r = max(r_begin, int64_t(0)); r < min(r_end, rows); ++r) {
              int64_t from = r;
              if (slots != nullptr) from = slots[r] >= 0 ? slots[r] / top_k : -1;
              if (from < 0 || from >= x_rows || col >= d) continue;
              const uint32_t v = static_cast<uint32_t>(x[from * d + col + c] & 0x7fffu) << 16;
              if (v <= kInfBits) top[c] = max(top[c], v);
            }
          }
        }
        int ex[4];
        uint32_t inv[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          ex[c] = scale_exponent(top[c]);
          inv[c] = inverse_scale_bf16(ex[c]);
        }
        const uint32_t inv01 = inv[0] | (inv[1] << 16), inv23 = inv[2] | (inv[3] << 16);
        if (any) {
#pragma unroll
          for (int r = 0; r < 16; ++r) words[r] = bf16_to_e4m3x4(u[r].x, u[r].y, inv01, inv23);
        }
        if (warp == 0 && col < d) {
          const uint32_t bytes = static_cast<uint32_t>(ex[0] + 127) | (static_cast<uint32_t>(ex[1] + 127) << 8) |
                                 (static_cast<uint32_t>(ex[2] + 127) << 16) | (static_cast<uint32_t>(ex[3] + 127) << 24);
          *reinterpret_cast<uint32_t*>(scales + static_cast<int64_t>(b) * d + col) = bytes;
        }
      }
      if (any && stripe + 1 < stripe1) load(stripe + 1);
      if (warp * 16 < width) put_transposed(tile, words, warp, lane);
      __syncthreads();
      write_transposed(tile, qt + static_cast<int64_t>(c0) * cap + static_cast<int64_t>(b) * 128, cap,
                       min(128, d - c0), width);
      // No barrier here: the next stripe's writes to `tile` come after the
      // barrier that follows col_max, which every thread reaches after its
      // reads of `tile`; col_max was read before this stripe's second one.
    }
  }
}

}  // namespace

cudaError_t launch_fp8_quantize_rows(const uint16_t* x, int64_t tokens, int d, const int32_t* pos,
                                     int k, int64_t rows, const int32_t* live, uint8_t* q,
                                     uint8_t* scales, int* err, cudaStream_t s) {
  const int blocks = (d + kFp8Block - 1) / kFp8Block;
  const int64_t grid = (tokens * blocks * 8 + kRowThreads - 1) / kRowThreads;
  return launch_pdl(quantize_rows_kernel, dim3(static_cast<unsigned>(grid)), dim3(kRowThreads), 0, s,
                    x, tokens, d, blocks, pos, k, rows, live, q, scales, err);
}

cudaError_t launch_fp8_quantize_blocks(const void* w, bool bf16, int experts, int n, int k,
                                       uint8_t* q, uint8_t* scales, uint8_t* qt, uint8_t* scales_t,
                                       int* err, cudaStream_t s) {
  const int64_t grid = int64_t(experts) * ((n + 127) / 128) * ((k + 127) / 128);
  const dim3 g(static_cast<unsigned>(grid)), b(kTileThreads);
  if (bf16)
    return launch_pdl(quantize_blocks_bf16_kernel, g, b, 0, s, static_cast<const uint16_t*>(w), n, k, q,
                      scales, qt, scales_t, err);
  return launch_pdl(quantize_blocks_kernel, g, b, 0, s, w, n, k, q, scales, qt, scales_t,
                    err);
}

cudaError_t launch_fp8_quantize_cols(const uint16_t* x, int64_t x_rows, int d,
                                     const int32_t* offsets, int experts, const int32_t* slots,
                                     int top_k, int64_t rows, uint8_t* qt, int64_t cap,
                                     uint8_t* scales, int* err, int num_sms, cudaStream_t s) {
  const int64_t tiles = (cap / 128) * ((d + 127) / 128);
  int64_t grid = tiles < 3 * num_sms ? tiles : 3 * num_sms;   // three blocks per SM
  if (grid < 1) grid = 1;                          // no columns: rows in offsets are reported
  return launch_pdl(quantize_cols_kernel, dim3(static_cast<unsigned>(grid)), dim3(kTileThreads), 0, s,
                    x, x_rows, d, offsets, experts, slots, top_k, rows, qt, cap, scales, err);
}

}  // namespace muon
