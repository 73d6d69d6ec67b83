// moe_api.cpp -- host side of the mixture-of-experts entry points of
// include/muon.h: argument validation and the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "muon.h"
#include "handle.h"
#include "kernels.h"
#include "moe.h"

namespace {

using muon::kFp8Block;
using muon::kMaxDim;

muon_status_t fail(muon_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return static_cast<muon_status_t>(muon::report(st, buf));
}

muon_status_t launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MUON_OK;
  return fail(MUON_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

muon_status_t info_of(muon_handle_t h, muon::HandleInfo* out) {
  return static_cast<muon_status_t>(muon::handle_info(h, out));
}

// A device buffer of a call: where it is and how long, for the checks.
struct Buffer {
  const void* ptr;
  int64_t bytes;
  bool out;
  int align = 16;
};

// Every buffer present and aligned, no output overlapping another.
template <int N>
muon_status_t check_buffers(const Buffer (&b)[N]) {
  for (int i = 0; i < N; ++i) {
    if (b[i].bytes == 0) continue;               // not wanted
    if (b[i].ptr == nullptr) return fail(MUON_ERR_INVALID_ARG, "NULL buffer");
    if (reinterpret_cast<uintptr_t>(b[i].ptr) % static_cast<uintptr_t>(b[i].align) != 0)
      return fail(MUON_ERR_INVALID_ARG, "buffers must be %d-byte aligned", b[i].align);
  }
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < i; ++j) {
      if (b[i].bytes == 0 || b[j].bytes == 0 || !(b[i].out || b[j].out)) continue;
      const uintptr_t p = reinterpret_cast<uintptr_t>(b[i].ptr), q = reinterpret_cast<uintptr_t>(b[j].ptr);
      if (p < q + static_cast<uintptr_t>(b[j].bytes) && q < p + static_cast<uintptr_t>(b[i].bytes))
        return fail(MUON_ERR_INVALID_ARG, "an output overlaps another buffer");
    }
  return MUON_OK;
}

int64_t blocks_of(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

bool hidden_ok(int32_t d) { return d >= 16 && d <= kMaxDim && d % 16 == 0; }

// Slots, rows and offsets travel as int32; a grid dimension holds them too.
constexpr int64_t kMaxSlots = (int64_t(1) << 31) - (int64_t(1) << 20);

muon_status_t check_hidden(const char* name, int32_t d) {
  if (hidden_ok(d)) return MUON_OK;
  return fail(MUON_ERR_INVALID_ARG, "%s must be a multiple of 16 from 16 to %d (got %d)", name,
              kMaxDim, d);
}

muon_status_t check_experts(int32_t experts) {
  if (experts >= 1 && experts <= muon::kMoeMaxExperts) return MUON_OK;
  return fail(MUON_ERR_INVALID_ARG, "experts must be 1..%d (got %d)", muon::kMoeMaxExperts, experts);
}

muon_status_t check_slots(int64_t tokens, int32_t top_k) {
  if (top_k < 1 || top_k > muon::kMoeMaxTopK)
    return fail(MUON_ERR_INVALID_ARG, "top_k must be 1..%d (got %d)", muon::kMoeMaxTopK, top_k);
  if (tokens < 0 || tokens > kMaxSlots / top_k)       // the product may not fit 64 bits
    return fail(MUON_ERR_INVALID_ARG, "tokens out of range (%lld)", static_cast<long long>(tokens));
  return MUON_OK;
}

muon_status_t check_rows(int64_t rows) {
  if (rows >= 0 && rows <= kMaxSlots) return MUON_OK;
  return fail(MUON_ERR_INVALID_ARG, "rows out of range (%lld)", static_cast<long long>(rows));
}

muon_status_t check_dtype(int32_t type) {
  if (type == MUON_FP32 || type == MUON_BF16) return MUON_OK;
  return fail(MUON_ERR_INVALID_ARG, "unknown element type %d", type);
}

#define MUON_TRY(expr)                       \
  do {                                       \
    const muon_status_t st_ = (expr);        \
    if (st_ != MUON_OK) return st_;          \
  } while (0)

muon_status_t check_route(int64_t tokens, int32_t experts, int32_t top_k, int32_t type,
                          const muon_route_options_t* o) {
  MUON_TRY(check_experts(experts));
  MUON_TRY(check_slots(tokens, top_k));
  MUON_TRY(check_dtype(type));
  if (top_k > experts)
    return fail(MUON_ERR_INVALID_ARG, "top_k %d exceeds the %d experts", top_k, experts);
  if (o == nullptr) return fail(MUON_ERR_INVALID_ARG, "opts is NULL");
  if (o->score != MUON_SCORE_SIGMOID && o->score != MUON_SCORE_SOFTMAX)
    return fail(MUON_ERR_INVALID_ARG, "unknown score %d", o->score);
  if (!std::isfinite(o->scale)) return fail(MUON_ERR_INVALID_ARG, "scale must be finite");
  return MUON_OK;
}

}  // namespace

extern "C" {

muon_status_t muon_moe_route(muon_handle_t h, int64_t tokens, int32_t experts, int32_t top_k,
                             const void* logits, int32_t logits_type, const float* bias,
                             const uint8_t* mask, const muon_route_options_t* opts, int32_t* ids,
                             float* weights, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_route(tokens, experts, top_k, logits_type, opts));
  if (opts->groups < 1 || opts->groups > muon::kMoeMaxGroups || experts % opts->groups != 0)
    return fail(MUON_ERR_INVALID_ARG, "groups must be 1..%d and divide the %d experts (got %d)",
                muon::kMoeMaxGroups, experts, opts->groups);
  if (opts->top_groups < 1 || opts->top_groups > opts->groups)
    return fail(MUON_ERR_INVALID_ARG, "top_groups must be 1..groups (got %d)", opts->top_groups);
  if (opts->group_top != 1 && opts->group_top != 2)
    return fail(MUON_ERR_INVALID_ARG, "group_top must be 1 or 2 (got %d)", opts->group_top);
  if (top_k > opts->top_groups * (experts / opts->groups))
    return fail(MUON_ERR_INVALID_ARG, "top_k %d exceeds the experts of %d groups", top_k,
                opts->top_groups);
  if (tokens == 0) return MUON_OK;
  const int64_t el = logits_type == MUON_BF16 ? 2 : 4;
  MUON_TRY(check_buffers<5>({{logits, tokens * experts * el, false},
                             {bias, bias != nullptr ? int64_t(experts) * 4 : 0, false},
                             {mask, mask != nullptr ? tokens : 0, false, 1},
                             {ids, tokens * top_k * 4, true},
                             {weights, tokens * top_k * 4, true}}));
  muon::RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.mask = mask;
  a.ids = ids;
  a.weights = weights;
  a.tokens = tokens;
  a.experts = experts;
  a.k = top_k;
  a.softmax = opts->score == MUON_SCORE_SOFTMAX;
  // All groups chosen from: no groups.
  a.groups = opts->top_groups == opts->groups ? 1 : opts->groups;
  a.top_groups = opts->top_groups;
  const uint32_t size = static_cast<uint32_t>(experts / a.groups);
  a.group_size = static_cast<int32_t>(size);
  a.per_group = size == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + size - 1) / size);
  a.group_top = a.groups == 1 ? 1 : opts->group_top;
  a.renorm = opts->renormalize != 0;
  a.scale = opts->scale;
  a.err = hi.dev_err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_MOE_ROUTE, s);
  return launched(muon::launch_moe_route(a, logits_type == MUON_BF16, s), "route");
}

muon_status_t muon_moe_route_backward(muon_handle_t h, int64_t tokens, int32_t experts,
                                      int32_t top_k, const void* logits, int32_t logits_type,
                                      const int32_t* ids, const float* grad_weights,
                                      const muon_route_options_t* opts, void* grad_logits,
                                      void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_route(tokens, experts, top_k, logits_type, opts));
  if (tokens == 0) return MUON_OK;
  const int64_t el = logits_type == MUON_BF16 ? 2 : 4;
  MUON_TRY(check_buffers<4>({{logits, tokens * experts * el, false},
                             {ids, tokens * top_k * 4, false},
                             {grad_weights, tokens * top_k * 4, false},
                             {grad_logits, tokens * experts * el, true}}));
  muon::RouteArgs a{};
  a.logits = logits;
  a.ids = const_cast<int32_t*>(ids);
  a.grad = grad_weights;
  a.grad_logits = grad_logits;
  a.tokens = tokens;
  a.experts = experts;
  a.k = top_k;
  a.softmax = opts->score == MUON_SCORE_SOFTMAX;
  a.renorm = opts->renormalize != 0;
  a.scale = opts->scale;
  a.err = hi.dev_err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_MOE_ROUTE, s);
  return launched(muon::launch_moe_route_backward(a, logits_type == MUON_BF16, s), "route backward");
}

muon_status_t muon_moe_plan(muon_handle_t h, int64_t n_slots, int32_t experts, const int32_t* ids,
                            int32_t* offsets, int32_t* slots, int32_t* pos, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_experts(experts));
  MUON_TRY(check_rows(n_slots));
  MUON_TRY(check_buffers<4>({{ids, n_slots * 4, false},
                             {offsets, (int64_t(experts) + 1) * 4, true},
                             {slots, n_slots * 4, true},
                             {pos, n_slots * 4, true}}));
  void* scratch = nullptr;
  const size_t bytes = muon::moe_plan_scratch(n_slots, experts);
  if (bytes > 0)
    MUON_TRY(static_cast<muon_status_t>(muon::handle_scratch(h, bytes, &scratch)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int phase = 2 - muon::moe_plan_launches(n_slots); phase < 2; ++phase) {
    muon::LaunchMark mark(h, MUON_KERNEL_MOE_PLAN, s);
    MUON_TRY(launched(muon::launch_moe_plan(phase, ids, n_slots, experts, offsets, slots, pos,
                                            static_cast<int32_t*>(scratch), hi.dev_err, s),
                      "plan"));
  }
  return MUON_OK;
}

muon_status_t muon_moe_combine(muon_handle_t h, int64_t tokens, int32_t top_k, int64_t rows,
                               int32_t hidden, const uint16_t* y, const int32_t* pos,
                               const float* weights, uint16_t* out, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_slots(tokens, top_k));
  MUON_TRY(check_rows(rows));
  MUON_TRY(check_hidden("hidden", hidden));
  if (tokens == 0) return MUON_OK;
  MUON_TRY(check_buffers<4>({{y, rows * hidden * 2, false},
                             {pos, tokens * top_k * 4, false},
                             {weights, weights != nullptr ? tokens * top_k * 4 : 0, false},
                             {out, tokens * hidden * 2, true}}));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_MOE_COMBINE, s);
  return launched(muon::launch_moe_combine(y, pos, weights, out, tokens, top_k, hidden, rows,
                                           hi.dev_err, s),
                  "combine");
}

muon_status_t muon_moe_combine_backward(muon_handle_t h, int64_t tokens, int32_t top_k,
                                        int64_t rows, int32_t hidden, const uint16_t* grad_out,
                                        const uint16_t* y, const int32_t* pos,
                                        const float* weights, uint16_t* grad_y,
                                        float* grad_weights, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_slots(tokens, top_k));
  MUON_TRY(check_rows(rows));
  MUON_TRY(check_hidden("hidden", hidden));
  if (tokens == 0) return MUON_OK;
  MUON_TRY(check_buffers<6>(
      {{grad_out, tokens * hidden * 2, false},
       {y, grad_weights != nullptr ? rows * hidden * 2 : 0, false},
       {pos, tokens * top_k * 4, false},
       {weights, weights != nullptr ? tokens * top_k * 4 : 0, false},
       {grad_y, rows * hidden * 2, true},
       {grad_weights, grad_weights != nullptr ? tokens * top_k * 4 : 0, true}}));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_MOE_COMBINE, s);
  return launched(muon::launch_moe_combine_backward(grad_out, y, pos, weights, grad_y, grad_weights,
                                                    tokens, top_k, hidden, rows, hi.dev_err, s),
                  "combine backward");
}

muon_status_t muon_fp8_quantize_rows(muon_handle_t h, int64_t tokens, int32_t hidden,
                                     const uint16_t* x, const int32_t* pos, int32_t top_k,
                                     int64_t rows, const int32_t* live_rows, uint8_t* q,
                                     uint8_t* scales, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_hidden("hidden", hidden));
  if (pos != nullptr) {
    MUON_TRY(check_slots(tokens, top_k));
    MUON_TRY(check_rows(rows));
  } else {
    MUON_TRY(check_rows(tokens));
    rows = tokens;
  }
  const int64_t threads = tokens * blocks_of(hidden) * 8;
  if (threads / 256 >= (int64_t(1) << 31) - 1)
    return fail(MUON_ERR_INVALID_ARG, "x is too large for one call");
  if (tokens == 0) return MUON_OK;
  MUON_TRY(check_buffers<5>({{x, tokens * hidden * 2, false},
                             {pos, pos != nullptr ? tokens * top_k * 4 : 0, false},
                             {live_rows, live_rows != nullptr ? 4 : 0, false, 4},
                             {q, rows * hidden, true},
                             {scales, rows * blocks_of(hidden), true}}));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_FP8_QUANTIZE, s);
  return launched(muon::launch_fp8_quantize_rows(x, tokens, hidden, pos, top_k, rows, live_rows, q,
                                                 scales, hi.dev_err, s),
                  "row quantiser");
}

muon_status_t muon_fp8_quantize_blocks(muon_handle_t h, int32_t experts, int32_t n, int32_t k,
                                       const void* w, int32_t w_type, uint8_t* q, uint8_t* scales,
                                       uint8_t* qt, uint8_t* scales_t, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_dtype(w_type));
  MUON_TRY(check_hidden("n", n));
  MUON_TRY(check_hidden("k", k));
  if (experts < 0) return fail(MUON_ERR_INVALID_ARG, "experts < 0");
  if (int64_t(experts) * blocks_of(n) * blocks_of(k) >= (int64_t(1) << 31) - 1)
    return fail(MUON_ERR_INVALID_ARG, "w is too large for one call");
  if ((q == nullptr) != (scales == nullptr) || (qt == nullptr) != (scales_t == nullptr))
    return fail(MUON_ERR_INVALID_ARG, "values and scales come in pairs");
  if (q == nullptr && qt == nullptr) return fail(MUON_ERR_INVALID_ARG, "no output");
  if (experts == 0) return MUON_OK;
  const int64_t values = int64_t(experts) * n * k, sc = int64_t(experts) * blocks_of(n) * blocks_of(k);
  MUON_TRY(check_buffers<5>({{w, values * (w_type == MUON_BF16 ? 2 : 4), false},
                             {q, q != nullptr ? values : 0, true},
                             {scales, scales != nullptr ? sc : 0, true},
                             {qt, qt != nullptr ? values : 0, true},
                             {scales_t, scales_t != nullptr ? sc : 0, true}}));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_FP8_QUANTIZE, s);
  return launched(muon::launch_fp8_quantize_blocks(w, w_type == MUON_BF16, experts, n, k, q, scales,
                                                   qt, scales_t, hi.dev_err, s),
                  "block quantiser");
}

muon_status_t muon_fp8_quantize_cols(muon_handle_t h, int64_t x_rows, int32_t hidden,
                                     const uint16_t* x, int32_t experts, const int32_t* offsets,
                                     int64_t rows, const int32_t* slots, int32_t top_k, uint8_t* qt,
                                     int64_t capacity, uint8_t* scales, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_experts(experts));
  MUON_TRY(check_hidden("hidden", hidden));
  MUON_TRY(check_rows(rows));
  MUON_TRY(check_rows(x_rows));
  MUON_TRY(check_rows(capacity));
  if (capacity % kFp8Block != 0)
    return fail(MUON_ERR_INVALID_ARG, "capacity must be a multiple of 128");
  if (x_rows * (hidden / 16) >= (int64_t(1) << 32))
    return fail(MUON_ERR_INVALID_ARG, "x is too large for one call");
  if (slots != nullptr && (top_k < 1 || top_k > muon::kMoeMaxTopK))
    return fail(MUON_ERR_INVALID_ARG, "top_k must be 1..%d (got %d)", muon::kMoeMaxTopK, top_k);
  if (rows == 0) return MUON_OK;
  MUON_TRY(check_buffers<5>({{x, x_rows * hidden * 2, false},
                             {offsets, (int64_t(experts) + 1) * 4, false},
                             {slots, slots != nullptr ? rows * 4 : 0, false},
                             {qt, capacity * hidden, true},
                             {scales, capacity / kFp8Block * hidden, true}}));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_FP8_QUANTIZE, s);
  return launched(muon::launch_fp8_quantize_cols(x, x_rows, hidden, offsets, experts, slots, top_k,
                                                 rows, qt, capacity, scales, hi.dev_err, hi.num_sms,
                                                 s),
                  "column quantiser");
}

muon_status_t muon_fp8_grouped_matmul(muon_handle_t h, int64_t rows, int32_t experts, int32_t n,
                                      int32_t k, const uint8_t* x, const uint8_t* x_scales,
                                      const uint8_t* w, const uint8_t* w_scales,
                                      const int32_t* offsets, uint16_t* y, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_experts(experts));
  MUON_TRY(check_rows(rows));
  MUON_TRY(check_hidden("n", n));
  MUON_TRY(check_hidden("k", k));
  if (rows == 0) return MUON_OK;
  MUON_TRY(check_buffers<6>({{x, rows * k, false},
                             {x_scales, rows * blocks_of(k), false},
                             {w, int64_t(experts) * n * k, false},
                             {w_scales, int64_t(experts) * blocks_of(n) * blocks_of(k), false},
                             {offsets, (int64_t(experts) + 1) * 4, false},
                             {y, rows * n * 2, true}}));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_FP8_PRODUCT, s);
  return launched(muon::launch_fp8_grouped_matmul(x, x_scales, w, w_scales, offsets, experts, rows,
                                                  n, k, y, hi.dev_err, hi.fp8_pairs.matmul, s),
                  "grouped product");
}

muon_status_t muon_fp8_grouped_wgrad(muon_handle_t h, int32_t experts, int32_t n, int32_t k,
                                     int64_t capacity, const uint8_t* yt, const uint8_t* yt_scales,
                                     const uint8_t* xt, const uint8_t* xt_scales,
                                     const int32_t* offsets, float* dw, int32_t accumulate,
                                     void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_experts(experts));
  MUON_TRY(check_rows(capacity));
  MUON_TRY(check_hidden("n", n));
  MUON_TRY(check_hidden("k", k));
  if (capacity % kFp8Block != 0)
    return fail(MUON_ERR_INVALID_ARG, "capacity must be a multiple of 128");
  MUON_TRY(check_buffers<6>({{yt, capacity * n, false},
                             {yt_scales, capacity / kFp8Block * n, false},
                             {xt, capacity * k, false},
                             {xt_scales, capacity / kFp8Block * k, false},
                             {offsets, (int64_t(experts) + 1) * 4, false},
                             {dw, int64_t(experts) * n * k * 4, true}}));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_FP8_WGRAD, s);
  return launched(muon::launch_fp8_grouped_wgrad(yt, yt_scales, xt, xt_scales, offsets, experts,
                                                 capacity, n, k, dw, accumulate != 0, hi.dev_err,
                                                 hi.fp8_pairs.wgrad, s),
                  "weight gradient");
}

}  // extern "C"
