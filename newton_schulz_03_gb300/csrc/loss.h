// loss.h -- launch interface of the losses on logits (loss_api.cpp validates,
// k_loss.cu launches).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace muon {

constexpr int kLossMaxTargets = 1024;              // teacher's logits per token
constexpr int32_t kLossMaxVocab = 1 << 24;
constexpr int64_t kLossMaxTokens = int64_t(1) << 27;   // tokens x cluster is a grid's x

// Self-test of the waits, where rows are streamed: after each block's first row
// nothing brings the logits, or what else a row needs.
enum LossStall : int32_t { kLossStallNone = 0, kLossStallLogits = 1, kLossStallTargets = 2 };

struct LossArgs {
  const void* logits;          // [tokens], `ld` elements apart
  int64_t ld;
  void* grad_logits;           // the logits' type, `grad_ld` elements apart, or NULL
  int64_t grad_ld;
  int64_t tokens;
  int32_t vocab;
  const uint8_t* mask;         // [tokens] or NULL; 0: the token is left out
  float temperature, inv_temperature, log2e_over_t;
  float* loss;                 // [tokens]; backward alone: not used
  float* lse;                  // [tokens]: out, or (backward alone) in
  const float* grad_loss;      // [tokens]
  // distillation
  const void* teacher;         // [tokens][targets], FP32 or BF16
  int32_t teacher_bf16;
  const int32_t* ids;          // [tokens][targets]
  int32_t targets;
  float scale;
  // policy
  const int32_t* actions;      // [tokens]
  const float* advantages;
  const float* old_logp;       // or NULL
  const float* ref_logp;       // or NULL
  float* logp;                 // out, or (backward alone) in
  float ratio_low, ratio_high; // 1 - clip_low, 1 + clip_high
  float kl_coef;
  int* err;
  int32_t stall;               // LossStall
};

// Shared-memory attributes of the kernels (called when a handle is made, with its
// device current).
cudaError_t loss_init();

// grad: with the gradient; backward: from lse (and logp), without the loss.
cudaError_t launch_distill_loss(const LossArgs& a, bool bf16, bool grad, bool backward, int num_sms,
                                cudaStream_t s);
cudaError_t launch_policy_loss(const LossArgs& a, bool bf16, bool grad, bool backward, int num_sms,
                               cudaStream_t s);

}  // namespace muon
