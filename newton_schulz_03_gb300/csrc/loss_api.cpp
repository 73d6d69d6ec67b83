// loss_api.cpp -- host side of the losses on logits of include/muon.h:
// argument validation and the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "muon.h"
#include "checks.h"
#include "handle.h"
#include "kernels.h"
#include "loss.h"

namespace {

using namespace muon::checks;

constexpr int64_t kMaxPitch = int64_t(1) << 31;

muon_status_t check_temperature(float t) {
  // 1 / t, and so log2(e) / t, are ordinary numbers.
  if (t >= 1e-4f && t <= 1e4f) return MUON_OK;
  return fail(MUON_ERR_INVALID_ARG, "temperature must be 1e-4 to 1e4 (got %g)", static_cast<double>(t));
}

muon_status_t check_sizes(int64_t tokens, int32_t vocab, int32_t type, int64_t ld) {
  MUON_TRY(check_dtype(type));
  if (tokens < 0 || tokens > muon::kLossMaxTokens)
    return fail(MUON_ERR_INVALID_ARG, "tokens out of range (%lld)", static_cast<long long>(tokens));
  if (vocab < 1 || vocab > muon::kLossMaxVocab)
    return fail(MUON_ERR_INVALID_ARG, "vocab must be 1..%d (got %d)", muon::kLossMaxVocab, vocab);
  if (ld < vocab || ld > kMaxPitch)
    return fail(MUON_ERR_INVALID_ARG, "a pitch must be vocab (%d) to 2^31 (got %lld)", vocab,
                static_cast<long long>(ld));
  return MUON_OK;
}

int64_t extent(int64_t tokens, int32_t vocab, int64_t ld, int64_t el) {
  return ((tokens - 1) * ld + vocab) * el;
}

// The logits and their gradient: apart, or the same rows (the gradient then
// takes the logits' place).  Leaves in *logits_bytes what is still to be
// compared with the other buffers: nothing where the gradient stands for both.
muon_status_t check_gradient(const muon::LossArgs& a, int64_t el, bool grad, int64_t* logits_bytes) {
  *logits_bytes = extent(a.tokens, a.vocab, a.ld, el);
  if (grad && a.grad_logits == a.logits && a.grad_logits != nullptr) {
    if (a.grad_ld != a.ld)
      return fail(MUON_ERR_INVALID_ARG, "a gradient in place of the logits has their pitch");
    *logits_bytes = 0;
  }
  return MUON_OK;
}

int64_t per_token(const void* p, int64_t tokens) { return p != nullptr ? tokens * 4 : 0; }

muon_status_t distill(muon_handle_t h, int64_t tokens, int32_t vocab, const void* logits,
                      int32_t logits_type, int64_t ld, int32_t targets, const void* teacher,
                      int32_t teacher_type, const int32_t* ids, const uint8_t* mask,
                      const muon_distill_options_t* o, float* loss, float* lse,
                      const float* grad_loss, void* grad_logits, int64_t grad_ld, bool grad,
                      bool backward, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_sizes(tokens, vocab, logits_type, ld));
  if (grad) MUON_TRY(check_sizes(tokens, vocab, logits_type, grad_ld));
  MUON_TRY(check_dtype(teacher_type));
  if (targets < 1 || targets > muon::kLossMaxTargets)
    return fail(MUON_ERR_INVALID_ARG, "targets must be 1..%d (got %d)", muon::kLossMaxTargets, targets);
  if (o == nullptr) return fail(MUON_ERR_INVALID_ARG, "opts is NULL");
  MUON_TRY(check_temperature(o->temperature));
  if (!std::isfinite(o->scale)) return fail(MUON_ERR_INVALID_ARG, "scale must be finite");
  if (tokens == 0) return MUON_OK;
  const int64_t el = logits_type == MUON_BF16 ? 2 : 4, tel = teacher_type == MUON_BF16 ? 2 : 4;
  muon::LossArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.grad_logits = grad_logits;
  a.grad_ld = grad_ld;
  a.tokens = tokens;
  a.vocab = vocab;
  a.mask = mask;
  a.temperature = o->temperature;
  a.inv_temperature = 1.0f / o->temperature;
  a.log2e_over_t = static_cast<float>(1.4426950408889634 / static_cast<double>(o->temperature));
  a.loss = loss;
  a.lse = lse;
  a.grad_loss = grad_loss;
  a.teacher = teacher;
  a.teacher_bf16 = teacher_type == MUON_BF16;
  a.ids = ids;
  a.targets = targets;
  a.scale = o->scale;
  a.err = hi.dev_err;
  int64_t logits_bytes;
  MUON_TRY(check_gradient(a, el, grad, &logits_bytes));
  MUON_TRY(check_buffers<8>(
      {{logits, logits_bytes, false, static_cast<int>(el)},
       {teacher, tokens * targets * tel, false, static_cast<int>(tel)},
       {ids, tokens * targets * 4, false, 4},
       {mask, mask != nullptr ? tokens : 0, false, 1},
       {loss, backward ? 0 : tokens * 4, true, 4},
       {lse, tokens * 4, !backward, 4},
       {grad_loss, grad ? tokens * 4 : 0, false, 4},
       {grad_logits, grad ? extent(tokens, vocab, grad_ld, el) : 0, true, static_cast<int>(el)}}));
  if (grad && !backward) a.stall = muon::take_loss_stall(h);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_LOSS, s);
  return launched(muon::launch_distill_loss(a, logits_type == MUON_BF16, grad, backward, hi.num_sms, s),
                  "distillation loss");
}

muon_status_t policy(muon_handle_t h, int64_t tokens, int32_t vocab, const void* logits,
                     int32_t logits_type, int64_t ld, const int32_t* actions,
                     const float* advantages, const float* old_logp, const float* ref_logp,
                     const uint8_t* mask, const muon_policy_options_t* o, float* loss, float* logp,
                     float* lse, const float* grad_loss, void* grad_logits, int64_t grad_ld,
                     bool grad, bool backward, void* stream) {
  muon::HandleInfo hi;
  MUON_TRY(info_of(h, &hi));
  MUON_TRY(check_sizes(tokens, vocab, logits_type, ld));
  if (grad) MUON_TRY(check_sizes(tokens, vocab, logits_type, grad_ld));
  if (o == nullptr) return fail(MUON_ERR_INVALID_ARG, "opts is NULL");
  MUON_TRY(check_temperature(o->temperature));
  if (!(o->clip_low >= 0.0f && o->clip_low <= 1.0f) || !(o->clip_high >= 0.0f) ||
      !std::isfinite(o->clip_high))
    return fail(MUON_ERR_INVALID_ARG, "clip_low must be 0 to 1 and clip_high 0 or more");
  if (!std::isfinite(o->kl_coef)) return fail(MUON_ERR_INVALID_ARG, "kl_coef must be finite");
  if (tokens == 0) return MUON_OK;
  const int64_t el = logits_type == MUON_BF16 ? 2 : 4;
  muon::LossArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.grad_logits = grad_logits;
  a.grad_ld = grad_ld;
  a.tokens = tokens;
  a.vocab = vocab;
  a.mask = mask;
  a.temperature = o->temperature;
  a.inv_temperature = 1.0f / o->temperature;
  a.log2e_over_t = static_cast<float>(1.4426950408889634 / static_cast<double>(o->temperature));
  a.loss = loss;
  a.lse = lse;
  a.logp = logp;
  a.grad_loss = grad_loss;
  a.actions = actions;
  a.advantages = advantages;
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.ratio_low = 1.0f - o->clip_low;
  a.ratio_high = 1.0f + o->clip_high;
  a.kl_coef = o->kl_coef;
  a.err = hi.dev_err;
  int64_t logits_bytes;
  MUON_TRY(check_gradient(a, el, grad, &logits_bytes));
  MUON_TRY(check_buffers<11>(
      {{logits, logits_bytes, false, static_cast<int>(el)},
       {actions, tokens * 4, false, 4},
       {advantages, tokens * 4, false, 4},
       {old_logp, per_token(old_logp, tokens), false, 4},
       {ref_logp, per_token(ref_logp, tokens), false, 4},
       {mask, mask != nullptr ? tokens : 0, false, 1},
       {loss, backward ? 0 : tokens * 4, true, 4},
       {logp, tokens * 4, !backward, 4},
       {lse, tokens * 4, !backward, 4},
       {grad_loss, grad ? tokens * 4 : 0, false, 4},
       {grad_logits, grad ? extent(tokens, vocab, grad_ld, el) : 0, true, static_cast<int>(el)}}));
  if (grad && !backward) a.stall = muon::take_loss_stall(h);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  muon::LaunchMark mark(h, MUON_KERNEL_LOSS, s);
  return launched(muon::launch_policy_loss(a, logits_type == MUON_BF16, grad, backward, hi.num_sms, s),
                  "policy loss");
}

}  // namespace

extern "C" {

muon_status_t muon_distill_loss(muon_handle_t h, int64_t tokens, int32_t vocab, const void* logits,
                                int32_t logits_type, int64_t ld, int32_t targets,
                                const void* teacher, int32_t teacher_type, const int32_t* ids,
                                const uint8_t* mask, const muon_distill_options_t* opts,
                                float* loss, float* lse, const float* grad_loss, void* grad_logits,
                                int64_t grad_ld, void* stream) {
  return distill(h, tokens, vocab, logits, logits_type, ld, targets, teacher, teacher_type, ids, mask,
                 opts, loss, lse, grad_loss, grad_logits, grad_ld,
                 grad_loss != nullptr || grad_logits != nullptr, false, stream);
}

muon_status_t muon_distill_loss_backward(muon_handle_t h, int64_t tokens, int32_t vocab,
                                         const void* logits, int32_t logits_type, int64_t ld,
                                         int32_t targets, const void* teacher, int32_t teacher_type,
                                         const int32_t* ids, const uint8_t* mask,
                                         const muon_distill_options_t* opts, const float* lse,
                                         const float* grad_loss, void* grad_logits,
                                         int64_t grad_ld, void* stream) {
  return distill(h, tokens, vocab, logits, logits_type, ld, targets, teacher, teacher_type, ids, mask,
                 opts, nullptr, const_cast<float*>(lse), grad_loss, grad_logits, grad_ld, true, true,
                 stream);
}

muon_status_t muon_policy_loss(muon_handle_t h, int64_t tokens, int32_t vocab, const void* logits,
                               int32_t logits_type, int64_t ld, const int32_t* actions,
                               const float* advantages, const float* old_logp,
                               const float* ref_logp, const uint8_t* mask,
                               const muon_policy_options_t* opts, float* loss, float* logp,
                               float* lse, const float* grad_loss, void* grad_logits,
                               int64_t grad_ld, void* stream) {
  return policy(h, tokens, vocab, logits, logits_type, ld, actions, advantages, old_logp, ref_logp, mask,
                opts, loss, logp, lse, grad_loss, grad_logits, grad_ld,
                grad_loss != nullptr || grad_logits != nullptr, false, stream);
}

muon_status_t muon_policy_loss_backward(muon_handle_t h, int64_t tokens, int32_t vocab,
                                        const void* logits, int32_t logits_type, int64_t ld,
                                        const int32_t* actions, const float* advantages,
                                        const float* old_logp, const float* ref_logp,
                                        const uint8_t* mask, const muon_policy_options_t* opts,
                                        const float* logp, const float* lse, const float* grad_loss,
                                        void* grad_logits, int64_t grad_ld, void* stream) {
  return policy(h, tokens, vocab, logits, logits_type, ld, actions, advantages, old_logp, ref_logp, mask,
                opts, nullptr, const_cast<float*>(logp), const_cast<float*>(lse), grad_loss, grad_logits,
                grad_ld, true, true, stream);
}

}  // extern "C"
