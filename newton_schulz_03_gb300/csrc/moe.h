// moe.h -- launch interface of the mixture-of-experts kernels
// (moe_api.cpp validates, the CUDA translation units launch).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace muon {

// ------------------------------------------------------------------ routing
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;
constexpr int kMoeMaxGroups = 32;

struct RouteArgs {
  const void* logits;      // [tokens][experts], FP32 or BF16
  const float* bias;       // [experts] or NULL
  const uint8_t* mask;     // [tokens] or NULL; 0: the token has no experts
  int32_t* ids;            // [tokens][k]
  float* weights;          // forward: out [tokens][k]
  const float* grad;       // backward: [tokens][k]
  void* grad_logits;       // backward: [tokens][experts], the logits' type
  int64_t tokens;
  int32_t experts, k;
  int32_t softmax;         // 0: sigmoid scores
  int32_t groups, top_groups, group_top;
  int32_t group_size;      // experts per group
  uint32_t per_group;      // ceil(2^32 / experts per group): i * it >> 32 is i's group
  int32_t renorm;
  float scale;
  int* err;
};

cudaError_t launch_moe_route(const RouteArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_moe_route_backward(const RouteArgs& a, bool bf16, cudaStream_t s);

// ------------------------------------------------------------------ grouping
// Scratch (bytes) of the plan of n slots over `experts` experts (0: none).
size_t moe_plan_scratch(int64_t n, int experts);
// Kernel launches it makes.
int moe_plan_launches(int64_t n);
// phase 0: the chunks' histograms (only when moe_plan_launches(n) == 2);
// phase 1: offsets, slots and pos.
cudaError_t launch_moe_plan(int phase, const int32_t* ids, int64_t n, int experts,
                            int32_t* offsets, int32_t* slots, int32_t* pos, int32_t* scratch,
                            int* err, cudaStream_t s);

cudaError_t launch_moe_combine(const uint16_t* y, const int32_t* pos, const float* w,
                               uint16_t* out, int64_t tokens, int k, int d, int64_t rows, int* err,
                               cudaStream_t s);
cudaError_t launch_moe_combine_backward(const uint16_t* grad_out, const uint16_t* y,
                                        const int32_t* pos, const float* w, uint16_t* grad_y,
                                        float* grad_w, int64_t tokens, int k, int d, int64_t rows,
                                        int* err, cudaStream_t s);

// ------------------------------------------------------------------ FP8
// CTA pairs of the products' persistent grids on a handle's device.
struct Fp8Pairs {
  int matmul, wgrad;
};

// Pairs of such a grid: what `query` (an int* to how many clusters the GPU
// holds at once) says, at most one pair per two SMs.  A query that fails, or
// finds no room, is an error and leaves *out alone.
template <typename Query>
cudaError_t resident_pairs(Query query, int num_sms, int* out) {
  int n = 0;
  const cudaError_t e = query(&n);
  if (e != cudaSuccess) return e;
  if (n < 1 || num_sms < 2) return cudaErrorInvalidConfiguration;
  *out = n < num_sms / 2 ? n : num_sms / 2;
  return cudaSuccess;
}

// Shared-memory attributes of the kernels, and the products' pairs (called
// when a handle is made, with its device current).
cudaError_t moe_plan_init();
cudaError_t fp8_gemm_init(int num_sms, Fp8Pairs* pairs);

constexpr int kFp8Block = 128;   // values that share one scale

// x [tokens][d] BF16 -> q e4m3, scales E8M0 [.][ceil(d/128)].  pos NULL:
// row t goes to row t; else to every row pos[t][j] >= 0 (of `rows`).  live:
// NULL, or how many rows of x there are.
cudaError_t launch_fp8_quantize_rows(const uint16_t* x, int64_t tokens, int d, const int32_t* pos,
                                     int k, int64_t rows, const int32_t* live, uint8_t* q,
                                     uint8_t* scales, int* err, cudaStream_t s);

// w [experts][n][k], FP32 or BF16 -> q [experts][n][k] and qt
// [experts][k][n] with one scale per 128 x 128 block; either output may be NULL.
cudaError_t launch_fp8_quantize_blocks(const void* w, bool bf16, int experts, int n, int k,
                                       uint8_t* q, uint8_t* scales, uint8_t* qt, uint8_t* scales_t,
                                       int* err, cudaStream_t s);

// Rows [offsets[e], offsets[e+1]) of each expert, 128 at a time: qt [d][cap]
// and scales [cap / 128][d], an expert's columns starting at a multiple of
// 128, zero from its rows to the next multiple of 32 (not written past that).  Row r is x[r], or x[slots[r] / top_k].
// `rows`: how many rows offsets may reach.
cudaError_t launch_fp8_quantize_cols(const uint16_t* x, int64_t x_rows, int d,
                                     const int32_t* offsets, int experts, const int32_t* slots,
                                     int top_k, int64_t rows, uint8_t* qt, int64_t cap,
                                     uint8_t* scales, int* err, int num_sms, cudaStream_t s);

// y[r] = x[r] w[e]^T for the rows of each expert: x e4m3 [rows][k] with
// scales [rows][kb], w e4m3 [experts][n][k] with scales [experts][nb][kb]
// (nb, kb: blocks of 128), y BF16 [rows][n].
cudaError_t launch_fp8_grouped_matmul(const uint8_t* x, const uint8_t* x_scales, const uint8_t* w,
                                      const uint8_t* w_scales, const int32_t* offsets, int experts,
                                      int64_t rows, int n, int k, uint16_t* y, int* err, int pairs,
                                      cudaStream_t s);

// dw[e] (+)= the expert's columns of yt times those of xt transposed: yt
// e4m3 [n][cap], scales [cap / 128][n]; xt [k][cap], [cap / 128][k]; dw FP32
// [experts][n][k].
cudaError_t launch_fp8_grouped_wgrad(const uint8_t* yt, const uint8_t* yt_scales,
                                     const uint8_t* xt, const uint8_t* xt_scales,
                                     const int32_t* offsets, int experts, int64_t cap, int n, int k,
                                     float* dw, bool accumulate, int* err, int pairs,
                                     cudaStream_t s);

}  // namespace muon
