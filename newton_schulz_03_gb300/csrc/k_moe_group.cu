// k_moe_group.cu -- grouping of (token, choice) slots by expert, and the
// weighted sum of the experts' rows back into tokens, with its backward pass.
//
// Plan: slot i = t k + j holds expert ids[t][j].  Rows are the slots in order
// of expert, then of slot (a stable counting sort): offsets[e] the first row
// of expert e, slots[r] the slot of row r, pos[i] the row of slot i.  Slots
// without an expert (-1) get no row.  The order is a function of ids alone:
// no atomics decide a rank.
//   Chunks of Q x 1024 slots, one block each: chunk histograms (one launch), then
// every block sums the histograms before its own and ranks its slots (second
// launch).  Up to 2048 slots, one block does all of it in one launch: the
// serving case, where a launch costs as much as the work.  Bound by latency: Q
// is the least of 1, 2, 4, 8 that keeps to 128 chunks, whose histograms a thread
// sums sixteen loads at a time.  57337 slots over 512 experts take 8.2 us (14
// chunks of 4096: 12.7 us), 458752 slots 16 us, 259 slots 2.4 us.  Past 2^20 slots
// there are more than 128 chunks, and their sums cost the square of the number:
// 2^20 slots 31 us from a cold cache, 2^22 132 us, 2^24 0.9 ms, 2^26 11 ms.
//
// Combine: out[t] = sum_j w[t][j] y[pos[t][j]], FP32 sums in the order of j,
// rounded once.  Backward: grad_y[pos[t][j]] = w[t][j] grad_out[t] and
// grad_w[t][j] = <grad_out[t], y[pos[t][j]]>.  One block per token, 16 bytes
// per thread and load, four rows' loads in flight together: bound by HBM (k rows
// of y per token; backward reads and writes them).  8191 tokens x 7 rows of 4096:
// 79 us forward (6.8 TB/s), 150 us backward.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "launch.cuh"
#include "moe.h"

namespace muon {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kOneBlock = 2048;                     // slots that one block takes alone
constexpr int kMaxChunks = 128;                     // as long as Q <= 8 allows

// Q of n slots: a block takes Q * 1024.
int plan_q(int64_t n) {
  int q = 1;
  while (q < 8 && int64_t(q) * kPlanThreads * (n <= kOneBlock ? 1 : kMaxChunks) < n) q *= 2;
  return q;
}
int64_t plan_chunks(int64_t n) {
  const int64_t chunk = int64_t(plan_q(n)) * kPlanThreads;
  return n > 0 ? (n + chunk - 1) / chunk : 1;
}

// Expert of a slot, or -1; anything else is reported and counts as none.
__device__ __forceinline__ int slot_expert(const int32_t* ids, int64_t i, int64_t n, int experts,
                                           int* err) {
  if (i >= n) return -1;
  const int e = ids[i];
  if (e >= experts || e < -1) {
    atomicOr(err, kDevErrIndex);
    return -1;
  }
  return e;
}

template <int Q>
__global__ void __launch_bounds__(kPlanThreads) plan_histogram_kernel(
    const int32_t* __restrict__ ids, int64_t n, int experts, int32_t* __restrict__ hist, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int32_t count[kMoeMaxExperts];
  for (int e = threadIdx.x; e < experts; e += kPlanThreads) count[e] = 0;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * Q * kPlanThreads;
  int e[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q)
    e[q] = slot_expert(ids, i0 + q * kPlanThreads + threadIdx.x, n, experts, err);
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (e[q] >= 0) atomicAdd(&count[e[q]], 1);      // counts: any order
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kPlanThreads)
    hist[static_cast<int64_t>(blockIdx.x) * experts + e] = count[e];
}

// One block per chunk.  hist == NULL: the only chunk.
template <int Q>
__global__ void __launch_bounds__(kPlanThreads) plan_rank_kernel(
    const int32_t* __restrict__ ids, int64_t n, int experts, const int32_t* __restrict__ hist,
    int32_t* __restrict__ offsets, int32_t* __restrict__ slots, int32_t* __restrict__ pos,
    int* err) {
  extern __shared__ uint8_t plan_smem[];
  // [warp][expert] counts of the warp's slots, then their prefix over warps.
  uint16_t* wcount = reinterpret_cast<uint16_t*>(plan_smem);
  __shared__ int32_t base[kMoeMaxExperts];
  __shared__ int32_t warp_total[kPlanWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * experts / 2 + 1; i += kPlanThreads)
    reinterpret_cast<uint32_t*>(wcount)[i] = 0u;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();

  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kPlanWarps + warp) * Q * 32 + lane;
  int e[Q], rank[Q];
  uint16_t* mine = wcount + warp * experts;
#pragma unroll
  for (int q = 0; q < Q; ++q) e[q] = slot_expert(ids, i0 + q * 32, n, experts, err);
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const uint32_t same = __match_any_sync(kAll, e[q]);
    const int before = e[q] >= 0 ? mine[e[q]] : 0;
    rank[q] = before + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e[q] >= 0 && lane == __ffs(same) - 1) mine[e[q]] = static_cast<uint16_t>(before + __popc(same));
    __syncwarp();
  }
  __syncthreads();

  // Thread x stands for expert x (at most 1024 of them): counts of all
  // chunks and of those before this one, and the warps' prefix.
  const int x = threadIdx.x;
  int total = 0, earlier = 0;
  if (x < experts) {
    int sum = 0;
    for (int w0 = 0; w0 < kPlanWarps; w0 += 16) {
      int c[16];
#pragma unroll
      for (int w = 0; w < 16; ++w) c[w] = wcount[(w0 + w) * experts + x];
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        wcount[(w0 + w) * experts + x] = static_cast<uint16_t>(sum);
        sum += c[w];
      }
    }
    if (hist == nullptr) {
      total = sum;
    } else {
      const int b = static_cast<int>(blockIdx.x);
#pragma unroll 16
      for (int c = 0; c < static_cast<int>(gridDim.x); ++c) {
        const int v = hist[static_cast<int64_t>(c) * experts + x];
        total += v;
        earlier += c < b ? v : 0;
      }
    }
  }
  int incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = warp_total[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kAll, v, o);
      if (lane >= o) v += u;
    }
    warp_total[lane] = v;
  }
  __syncthreads();
  const int start = incl - total + (warp > 0 ? warp_total[warp - 1] : 0);
  if (x < experts) {
    base[x] = start + earlier;
    if (blockIdx.x == 0) offsets[x] = start;
  }
  const int all = warp_total[kPlanWarps - 1];
  if (blockIdx.x == 0 && x == 0) offsets[experts] = all;
  __syncthreads();

#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int64_t i = i0 + q * 32;
    if (i >= n) continue;
    int r = -1;
    if (e[q] >= 0) {
      r = base[e[q]] + mine[e[q]] + rank[q];
      slots[r] = static_cast<int32_t>(i);
    }
    pos[i] = r;
    if (i >= all) slots[i] = -1;                    // rows past the last one
  }
}

// ------------------------------------------------------------------ combine
constexpr int kCombineThreads = 256;
constexpr int kUnroll = 4;                          // rows in flight per thread

__device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
  f[0] = lo(u.x); f[1] = hi(u.x); f[2] = lo(u.y); f[3] = hi(u.y);
  f[4] = lo(u.z); f[5] = hi(u.z); f[6] = lo(u.w); f[7] = hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
}

// Rows and weights of one token, in shared memory; a row out of range is
// reported and counts as none.
__device__ __forceinline__ void load_choices(const int32_t* pos, const float* w, int64_t t, int k,
                                             int64_t rows, int* err, int32_t* row_s, float* w_s) {
  if (threadIdx.x < k) {
    int r = pos[t * k + threadIdx.x];
    if (r >= rows || r < -1) {
      atomicOr(err, kDevErrIndex);
      r = -1;
    }
    row_s[threadIdx.x] = r;
    w_s[threadIdx.x] = w != nullptr ? w[t * k + threadIdx.x] : 1.0f;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kCombineThreads) combine_kernel(
    const uint4* __restrict__ y, const int32_t* __restrict__ pos, const float* __restrict__ w,
    uint4* __restrict__ out, int k, int vecs, int64_t rows, int* err) {
  __shared__ int32_t row_s[kMoeMaxTopK];
  __shared__ float w_s[kMoeMaxTopK];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  load_choices(pos, w, t, k, rows, err, row_s, w_s);
  for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < k; j0 += kUnroll) {
      uint4 u[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int r = j0 + j < k ? row_s[j0 + j] : -1;
        u[j] = r >= 0 ? __ldcs(y + static_cast<int64_t>(r) * vecs + v) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        if (j0 + j >= k || row_s[j0 + j] < 0) continue;
        float f[8];
        unpack(u[j], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = fmaf(w_s[j0 + j], f[q], acc[q]);
      }
    }
    out[t * vecs + v] = pack8(acc);
  }
}

__global__ void __launch_bounds__(kCombineThreads) combine_backward_kernel(
    const uint4* __restrict__ grad_out, const uint4* __restrict__ y,
    const int32_t* __restrict__ pos, const float* __restrict__ w, uint4* __restrict__ grad_y,
    float* __restrict__ grad_w, int k, int vecs, int64_t rows, int* err) {
  __shared__ int32_t row_s[kMoeMaxTopK];
  __shared__ float w_s[kMoeMaxTopK];
  __shared__ float part[kCombineThreads / 32][kMoeMaxTopK];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  load_choices(pos, w, t, k, rows, err, row_s, w_s);
  for (int j0 = 0; j0 < k; j0 += kUnroll) {
    float dot[kUnroll] = {};
    for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
      uint4 u[kUnroll];
      const uint4 gu = grad_out[t * vecs + v];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int r = j0 + j < k ? row_s[j0 + j] : -1;
        u[j] = r >= 0 && grad_w != nullptr ? __ldcs(y + static_cast<int64_t>(r) * vecs + v)
                                           : make_uint4(0, 0, 0, 0);
      }
      float g[8];
      unpack(gu, g);
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int r = j0 + j < k ? row_s[j0 + j] : -1;
        if (r < 0) continue;
        float f[8], h[8];
        unpack(u[j], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          dot[j] = fmaf(g[q], f[q], dot[j]);
          h[q] = w_s[j0 + j] * g[q];
        }
        __stcs(grad_y + static_cast<int64_t>(r) * vecs + v, pack8(h));
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], o);
      if (lane == 0 && j0 + j < k) part[warp][j0 + j] = dot[j];
    }
  }
  if (grad_w == nullptr) return;
  __syncthreads();
  if (threadIdx.x < k) {
    float s = 0.f;
    for (int q = 0; q < static_cast<int>(blockDim.x >> 5); ++q) s += part[q][threadIdx.x];
    grad_w[t * k + threadIdx.x] = row_s[threadIdx.x] >= 0 ? s : 0.f;
  }
}

}  // namespace

namespace {
template <int Q>
cudaError_t plan_attr() {
  return cudaFuncSetAttribute(plan_rank_kernel<Q>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kPlanWarps * kMoeMaxExperts * 2 + 16);
}

template <int Q>
cudaError_t launch_plan(int phase, const int32_t* ids, int64_t n, int experts, int32_t* offsets,
                        int32_t* slots, int32_t* pos, int32_t* scratch, int* err, cudaStream_t s) {
  const int64_t chunks = plan_chunks(n);
  const dim3 grid(static_cast<unsigned>(chunks)), block(kPlanThreads);
  if (phase == 0)
    return launch_pdl(plan_histogram_kernel<Q>, grid, block, 0, s, ids, n, experts, scratch, err);
  return launch_pdl(plan_rank_kernel<Q>, grid, block, size_t(kPlanWarps) * experts * 2 + 16, s, ids,
                    n, experts, static_cast<const int32_t*>(chunks > 1 ? scratch : nullptr), offsets,
                    slots, pos, err);
}
}  // namespace

cudaError_t moe_plan_init() {
  cudaError_t e;
  if ((e = plan_attr<1>()) != cudaSuccess) return e;
  if ((e = plan_attr<2>()) != cudaSuccess) return e;
  if ((e = plan_attr<4>()) != cudaSuccess) return e;
  return plan_attr<8>();
}

size_t moe_plan_scratch(int64_t n, int experts) {
  const int64_t chunks = plan_chunks(n);
  return chunks > 1 ? size_t(chunks) * experts * 4 : 0;
}

int moe_plan_launches(int64_t n) { return plan_chunks(n) > 1 ? 2 : 1; }

cudaError_t launch_moe_plan(int phase, const int32_t* ids, int64_t n, int experts,
                            int32_t* offsets, int32_t* slots, int32_t* pos, int32_t* scratch,
                            int* err, cudaStream_t s) {
  switch (plan_q(n)) {
    case 1: return launch_plan<1>(phase, ids, n, experts, offsets, slots, pos, scratch, err, s);
    case 2: return launch_plan<2>(phase, ids, n, experts, offsets, slots, pos, scratch, err, s);
    case 4: return launch_plan<4>(phase, ids, n, experts, offsets, slots, pos, scratch, err, s);
    default: return launch_plan<8>(phase, ids, n, experts, offsets, slots, pos, scratch, err, s);
  }
}

cudaError_t launch_moe_combine(const uint16_t* y, const int32_t* pos, const float* w,
                               uint16_t* out, int64_t tokens, int k, int d, int64_t rows, int* err,
                               cudaStream_t s) {
  return launch_pdl(combine_kernel, dim3(static_cast<unsigned>(tokens)), dim3(kCombineThreads), 0,
                    s, reinterpret_cast<const uint4*>(y), pos, w, reinterpret_cast<uint4*>(out), k,
                    d / 8, rows, err);
}

cudaError_t launch_moe_combine_backward(const uint16_t* grad_out, const uint16_t* y,
                                        const int32_t* pos, const float* w, uint16_t* grad_y,
                                        float* grad_w, int64_t tokens, int k, int d, int64_t rows,
                                        int* err, cudaStream_t s) {
  return launch_pdl(combine_backward_kernel, dim3(static_cast<unsigned>(tokens)),
                    dim3(kCombineThreads), 0, s, reinterpret_cast<const uint4*>(grad_out),
                    reinterpret_cast<const uint4*>(y), pos, w, reinterpret_cast<uint4*>(grad_y),
                    grad_w, k, d / 8, rows, err);
}

}  // namespace muon
