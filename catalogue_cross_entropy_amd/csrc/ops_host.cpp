// C entry points of the operators around the losses (item embedding, log-probabilities
// over the catalogue, policy and preference losses): argument checks, then the launchers
// of k_embed.hip, k_logprob.hip and k_policy.hip.  Nothing here allocates or waits.
#include <hip/hip_runtime.h>

#include <cmath>

#include "rece_ops.h"

using namespace rece;

namespace {

constexpr int64_t I32_MAX = ((int64_t)1 << 31) - 1;

rece_status invalid(const char* msg) { return set_last_error(RECE_ERR_INVALID_ARGUMENT, msg); }
rece_status unsupported(const char* msg) { return set_last_error(RECE_ERR_UNSUPPORTED, msg); }

rece_status hip_status(hipError_t e) {
  return e == hipSuccess ? RECE_OK : set_last_error(RECE_ERR_HIP, hipGetErrorString(e));
}

bool misaligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

bool bad_dtype(int32_t t) { return t != RECE_F32 && t != RECE_BF16; }

rece_status check_embed(int64_t n, int64_t C, int32_t d) {
  if (n < 0 || C < 1 || d < 1) return invalid("n must be >= 0, C and d >= 1");
  if (n > I32_MAX || C > I32_MAX) return unsupported("n and C must fit in int32");
  if (d % 8 != 0 || d > 8192) return unsupported("d must be a multiple of 8, at most 8192");
  return RECE_OK;
}

rece_status check_logprob(int64_t s, int64_t C, int32_t d, int32_t dtype, uint32_t flags) {
  if (s < 1 || C < 1) return invalid("s and C must be >= 1");
  if (s > I32_MAX || C > I32_MAX) return unsupported("s and C must fit in int32");
  if (d != 32 && d != 64 && d != 128 && d != 256) return unsupported("d must be one of 32, 64, 128, 256");
  if (bad_dtype(dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (flags & ~(RECE_FLAG_BF16_GRADS | RECE_FLAG_NO_GRAD | RECE_FLAG_ENTROPY)) return invalid("unknown flag");
  return RECE_OK;
}

rece_status check_logprob_call(int64_t s, int64_t C, int32_t d, int32_t dtype, float temperature, uint32_t flags,
                               const void* X, const void* Y, const int32_t* ids, const void* ws, size_t ws_bytes) {
  const rece_status v = check_logprob(s, C, d, dtype, flags);
  if (v != RECE_OK) return v;
  // Below, a logit in base 2 may pass 2^31, where its float32 steps are beyond the range of the exponential that a
  // reference is taken out of; above, the values that stand for rows beyond the end come near 0.
  if (!(temperature >= 0x1p-20f && temperature <= 0x1p64f)) return invalid("temperature must be positive, from 2^-20 to 2^64");
  if (!X || !Y || !ids || !ws) return invalid("NULL input or workspace pointer");
  if (misaligned(X, 16) || misaligned(Y, 16) || misaligned(ws, 16)) return invalid("X, Y and workspace must be 16-byte aligned");
  if (misaligned(ids, 4)) return invalid("ids must be 4-byte aligned");
  if (ws_bytes < logprob_workspace_bytes(dtype == RECE_BF16, s, C, d, flags))
    return set_last_error(RECE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than rece_logprob_workspace_bytes");
  return RECE_OK;
}

rece_status check_policy(const rece_policy_config* c) {
  if (!c) return invalid("config is NULL");
  if (c->n < 0 || c->n_seq < 1) return invalid("n must be >= 0 and n_seq >= 1");
  if (c->n > I32_MAX || c->n_seq > I32_MAX - 1) return unsupported("n and n_seq must fit in int32");
  if (bad_dtype(c->dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (c->reduction != RECE_MEAN_TOKEN && c->reduction != RECE_MEAN_SEQUENCE) return invalid("unknown reduction");
  if (c->token_adv != 0 && c->token_adv != 1) return invalid("token_adv must be 0 or 1");
  if (!(c->clip_low >= 0.0f && c->clip_low <= 1.0f) || !(c->clip_high >= 0.0f) || !std::isfinite(c->clip_high))
    return invalid("clip_low must be in [0, 1] and clip_high >= 0");
  if (!std::isfinite(c->kl_coef) || !std::isfinite(c->entropy_coef)) return invalid("coefficients must be finite");
  return RECE_OK;
}

rece_status check_preference(const rece_preference_config* c) {
  if (!c) return invalid("config is NULL");
  if (c->n < 0 || c->n_seq < 1 || c->n_group < 1) return invalid("n must be >= 0, n_seq and n_group >= 1");
  if (c->n > I32_MAX || c->n_seq > I32_MAX - 1 || c->n_group > I32_MAX / 2)
    return unsupported("n and n_seq must fit in int32, n_group be at most 2^30 - 1");
  if (bad_dtype(c->dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (c->kind < RECE_PREF_SIGMOID || c->kind > RECE_PREF_SOFTMAX) return invalid("unknown kind");
  if (c->average != 0 && c->average != 1) return invalid("average must be 0 or 1");
  if (!(c->beta > 0.0f) || !std::isfinite(c->beta)) return invalid("beta must be positive and finite");
  if (!std::isfinite(c->margin)) return invalid("margin must be finite");
  if (!(c->smoothing >= 0.0f && c->smoothing < 1.0f)) return invalid("smoothing must be in [0, 1)");
  if (c->smoothing != 0.0f && c->kind != RECE_PREF_SIGMOID) return invalid("smoothing belongs to the sigmoid kind");
  return RECE_OK;
}

}  // namespace

extern "C" {

rece_status rece_embed_forward(void* stream, int64_t n, int64_t C, int32_t d, int32_t dtype, float scale,
                               const void* table, const int32_t* ids, void* out) {
  const rece_status v = check_embed(n, C, d);
  if (v != RECE_OK) return v;
  if (bad_dtype(dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (n == 0) return RECE_OK;
  if (!table || !ids || !out) return invalid("NULL pointer argument");
  if (misaligned(table, 16) || misaligned(out, 16) || misaligned(ids, 4))
    return invalid("table and out must be 16-byte aligned, ids 4-byte aligned");
  return hip_status(embed_forward(dtype == RECE_BF16, n, C, d, scale, table, ids, out, static_cast<hipStream_t>(stream)));
}

rece_status rece_embed_workspace_bytes(int64_t n, int64_t C, int32_t d, size_t* bytes) {
  const rece_status v = check_embed(n, C, d);
  if (v != RECE_OK) return v;
  if (!bytes) return invalid("bytes is NULL");
  *bytes = embed_workspace_bytes(n, C, d);
  return RECE_OK;
}

rece_status rece_embed_backward(void* stream, int64_t n, int64_t C, int32_t d, int32_t dtype, float scale,
                                uint32_t flags, const int32_t* ids, const void* dout, void* workspace,
                                size_t workspace_bytes, void* dtable) {
  const rece_status v = check_embed(n, C, d);
  if (v != RECE_OK) return v;
  if (bad_dtype(dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (flags & ~(RECE_FLAG_BF16_GRADS | RECE_FLAG_ACCUMULATE)) return invalid("unknown flag");
  const bool acc = flags & RECE_FLAG_ACCUMULATE, b16 = flags & RECE_FLAG_BF16_GRADS;
  if (acc && b16) return unsupported("gradients are accumulated in float32 only");
  if (!dtable || (n > 0 && (!ids || !dout || !workspace))) return invalid("NULL pointer argument");
  if (misaligned(dtable, 16) || (n > 0 && (misaligned(dout, 16) || misaligned(workspace, 16) || misaligned(ids, 4))))
    return invalid("dout, dtable and workspace must be 16-byte aligned, ids 4-byte aligned");
  if (n > 0 && workspace_bytes < embed_workspace_bytes(n, C, d))
    return set_last_error(RECE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than rece_embed_workspace_bytes");
  return hip_status(embed_backward(dtype == RECE_BF16, n, C, d, scale, b16, acc, ids, dout, workspace, dtable,
                                   static_cast<hipStream_t>(stream)));
}

rece_status rece_logprob_workspace_bytes(int64_t s, int64_t C, int32_t d, int32_t dtype, uint32_t flags, size_t* bytes) {
  const rece_status v = check_logprob(s, C, d, dtype, flags);
  if (v != RECE_OK) return v;
  if (!bytes) return invalid("bytes is NULL");
  *bytes = logprob_workspace_bytes(dtype == RECE_BF16, s, C, d, flags);
  return RECE_OK;
}

rece_status rece_logprob_forward(void* stream, int64_t s, int64_t C, int32_t d, int32_t dtype, float temperature,
                                 uint32_t flags, const void* X, const void* Y, const int32_t* ids, void* workspace,
                                 size_t workspace_bytes, float* logp, float* entropy) {
  const rece_status v = check_logprob_call(s, C, d, dtype, temperature, flags, X, Y, ids, workspace, workspace_bytes);
  if (v != RECE_OK) return v;
  if (!logp) return invalid("logp is NULL");
  if (!!(flags & RECE_FLAG_ENTROPY) != !!entropy) return invalid("entropy goes with RECE_FLAG_ENTROPY");
  if (misaligned(logp, 4) || misaligned(entropy, 4)) return invalid("logp and entropy must be 4-byte aligned");
  return hip_status(logprob_forward(dtype == RECE_BF16, s, C, d, temperature, flags, X, Y, ids, workspace, logp, entropy,
                                    static_cast<hipStream_t>(stream)));
}

rece_status rece_logprob_backward(void* stream, int64_t s, int64_t C, int32_t d, int32_t dtype, float temperature,
                                  uint32_t flags, const void* X, const void* Y, const int32_t* ids, void* workspace,
                                  size_t workspace_bytes, const float* dlogp, const float* dentropy, void* dX,
                                  void* dY) {
  const rece_status v = check_logprob_call(s, C, d, dtype, temperature, flags, X, Y, ids, workspace, workspace_bytes);
  if (v != RECE_OK) return v;
  if (flags & RECE_FLAG_NO_GRAD) return invalid("the forward call was made with RECE_FLAG_NO_GRAD");
  if (!dlogp || !dX || !dY) return invalid("NULL gradient pointer");
  if (dentropy && !(flags & RECE_FLAG_ENTROPY)) return invalid("dentropy needs RECE_FLAG_ENTROPY");
  if (misaligned(dX, 16) || misaligned(dY, 16) || misaligned(dlogp, 4) || misaligned(dentropy, 4))
    return invalid("dX and dY must be 16-byte aligned, dlogp and dentropy 4-byte aligned");
  return hip_status(logprob_backward(dtype == RECE_BF16, s, C, d, temperature, flags, X, Y, ids, workspace, dlogp,
                                     dentropy, dX, dY, static_cast<hipStream_t>(stream)));
}

rece_status rece_policy_workspace_bytes(const rece_policy_config* cfg, size_t* bytes) {
  const rece_status v = check_policy(cfg);
  if (v != RECE_OK) return v;
  if (!bytes) return invalid("bytes is NULL");
  *bytes = policy_workspace_bytes(*cfg);
  return RECE_OK;
}

rece_status rece_policy_loss(const rece_policy_config* cfg, void* stream, const void* logp, const void* old,
                             const void* ref, const void* entropy, const float* adv, const int32_t* offsets,
                             const uint8_t* mask, const float* dloss, void* workspace, size_t workspace_bytes,
                             float* loss, float* stats, void* dlogp, void* dentropy) {
  const rece_status v = check_policy(cfg);
  if (v != RECE_OK) return v;
  if (!offsets || !workspace || !loss || !stats) return invalid("NULL pointer argument");
  if (cfg->n > 0 && (!logp || !old || !adv)) return invalid("logp, old or adv is NULL");
  if (cfg->n > 0 && !ref && cfg->kl_coef != 0.0f) return invalid("kl_coef without ref");
  if (cfg->n > 0 && !entropy && cfg->entropy_coef != 0.0f) return invalid("entropy_coef without entropy");
  if (cfg->n > 0 && dentropy && !entropy) return invalid("dentropy without entropy");
  const unsigned ea = cfg->dtype == RECE_BF16 ? 2 : 4;
  if (misaligned(workspace, 16)) return invalid("workspace must be 16-byte aligned");
  for (const void* p : {logp, old, ref, entropy, static_cast<const void*>(dlogp), static_cast<const void*>(dentropy)})
    if (misaligned(p, ea)) return invalid("a token array is not aligned to its elements");
  for (const void* p : {static_cast<const void*>(adv), static_cast<const void*>(offsets), static_cast<const void*>(dloss),
                        static_cast<const void*>(loss), static_cast<const void*>(stats)})
    if (misaligned(p, 4)) return invalid("adv, offsets, dloss, loss and stats must be 4-byte aligned");
  if (workspace_bytes < policy_workspace_bytes(*cfg))
    return set_last_error(RECE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than rece_policy_workspace_bytes");
  return hip_status(policy_loss(*cfg, logp, old, ref, entropy, adv, offsets, mask, dloss, workspace, loss, stats, dlogp,
                                dentropy, static_cast<hipStream_t>(stream)));
}

rece_status rece_preference_workspace_bytes(const rece_preference_config* cfg, size_t* bytes) {
  const rece_status v = check_preference(cfg);
  if (v != RECE_OK) return v;
  if (!bytes) return invalid("bytes is NULL");
  *bytes = preference_workspace_bytes(*cfg);
  return RECE_OK;
}

rece_status rece_preference_loss(const rece_preference_config* cfg, void* stream, const void* logp, const void* ref,
                                 const int32_t* offsets, const int32_t* group_offsets, const uint8_t* mask,
                                 const float* dloss, void* workspace, size_t workspace_bytes, float* loss,
                                 float* loss_pg, float* rewards, void* dlogp) {
  const rece_status v = check_preference(cfg);
  if (v != RECE_OK) return v;
  if (!offsets || !group_offsets || !workspace || !loss || !loss_pg || !rewards) return invalid("NULL pointer argument");
  if (cfg->n > 0 && !logp) return invalid("logp is NULL");
  const unsigned ea = cfg->dtype == RECE_BF16 ? 2 : 4;
  if (misaligned(workspace, 16)) return invalid("workspace must be 16-byte aligned");
  for (const void* p : {logp, ref, static_cast<const void*>(dlogp)})
    if (misaligned(p, ea)) return invalid("a token array is not aligned to its elements");
  for (const void* p : {static_cast<const void*>(offsets), static_cast<const void*>(group_offsets),
                        static_cast<const void*>(dloss), static_cast<const void*>(loss),
                        static_cast<const void*>(loss_pg), static_cast<const void*>(rewards)})
    if (misaligned(p, 4)) return invalid("offsets, dloss and the outputs must be 4-byte aligned");
  if (workspace_bytes < preference_workspace_bytes(*cfg))
    return set_last_error(RECE_ERR_WORKSPACE_TOO_SMALL, "workspace smaller than rece_preference_workspace_bytes");
  return hip_status(preference_loss(*cfg, logp, ref, offsets, group_offsets, mask, dloss, workspace, loss, loss_pg,
                                    rewards, dlogp, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
