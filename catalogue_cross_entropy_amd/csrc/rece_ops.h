// Launchers of the operators around the losses and of the sequence encoder (ops_host.cpp and encoder_host.cpp call them).
// Apart from rece_internal.h, so that a change here is none of the loss kernels' sources.
#pragma once
#include "rece_internal.h"

namespace rece {

// Item embedding (k_embed.hip).
size_t embed_workspace_bytes(int64_t n, int64_t C, int d);
hipError_t embed_forward(bool bf16v, int64_t n, int64_t C, int d, float scale, const void* table, const int32_t* ids,
                         void* out, hipStream_t st);
hipError_t embed_backward(bool bf16v, int64_t n, int64_t C, int d, float scale, bool grad_bf16, bool accumulate,
                          const int32_t* ids, const void* dout, void* ws, void* dtable, hipStream_t st);
// Log-probabilities over the catalogue (k_logprob.hip).
size_t logprob_workspace_bytes(bool bf16v, int64_t s, int64_t C, int d, uint32_t flags);
hipError_t logprob_forward(bool bf16v, int64_t s, int64_t C, int d, float temperature, uint32_t flags, const void* X,
                           const void* Y, const int32_t* ids, void* ws, float* logp, float* entropy, hipStream_t st);
hipError_t logprob_backward(bool bf16v, int64_t s, int64_t C, int d, float temperature, uint32_t flags, const void* X,
                            const void* Y, const int32_t* ids, void* ws, const float* dlogp, const float* dentropy,
                            void* dX, void* dY, hipStream_t st);
// Losses on log-probabilities (k_policy.hip).
size_t policy_workspace_bytes(const rece_policy_config& c);
hipError_t policy_loss(const rece_policy_config& c, const void* logp, const void* old, const void* ref,
                       const void* entropy, const float* adv, const int32_t* offsets, const uint8_t* mask,
                       const float* dloss, void* ws, float* loss, float* stats, void* dlogp, void* dentropy,
                       hipStream_t st);
size_t preference_workspace_bytes(const rece_preference_config& c);
hipError_t preference_loss(const rece_preference_config& c, const void* logp, const void* ref, const int32_t* offsets,
                           const int32_t* group_offsets, const uint8_t* mask, const float* dloss, void* ws, float* loss,
                           float* loss_pg, float* rewards, void* dlogp, hipStream_t st);

// Attention over packed sequences, and of the last tokens over a cache (k_attention.hip).
size_t attention_workspace_bytes(const rece_attention_config& c);
hipError_t attention_forward(const rece_attention_config& c, const void* q, const void* k, const void* v,
                             const int32_t* offs, const float* bias, void* ws, void* out, hipStream_t st);
// strides: of dq, dk and dv rows, in elements
hipError_t attention_backward(const rece_attention_config& c, const void* q, const void* k, const void* v,
                              const int32_t* offs, const float* bias, const void* out, void* ws, const void* dout,
                              void* dq, void* dk, void* dv, float* dbias, const int64_t (&strides)[3], hipStream_t st);
size_t last_attention_workspace_bytes(const rece_attention_config& c, int64_t max_len);
hipError_t last_attention(const rece_attention_config& c, int64_t max_len, const void* q, const void* k, const void* v,
                          const int32_t* begin, const int32_t* length, const float* bias, void* ws, void* out,
                          hipStream_t st);
// Residual norm and rows in 8 bits (k_norm.hip).
hipError_t norm_forward(bool bf16v, int64_t n, int d, float eps, const void* x, const void* residual, const float* weight,
                        void* h, void* y, float* rstd, hipStream_t st);
hipError_t norm_forward_int8(bool bf16v, int64_t n, int d, float eps, const void* x, const void* residual,
                             const float* weight, void* h, int8_t* y8, float* scale, hipStream_t st);
hipError_t quantize_rows(bool bf16v, int64_t n, int d, const void* x, int8_t* x8, float* scale, hipStream_t st);
size_t norm_workspace_bytes(int64_t n, int d);
hipError_t norm_backward(bool bf16v, int64_t n, int d, const void* dy, const void* h, const void* dh, const float* weight,
                         const float* rstd, void* ws, void* dx, float* dweight, hipStream_t st);
// out[t] = sum over the rows of part[rows][cols], in a fixed order (float64 sums).
hipError_t launch_join_rows(const float* part, int rows, int cols, float* out, hipStream_t st);
// Scores of rows in 8 bits (k_int8.hip); int8_tiles: workgroups of the widest form.
int64_t int8_tiles(int64_t s, int64_t C);
hipError_t int8_scores(bool bf16v, int64_t s, int64_t C, int d, const int8_t* x, const float* sx, const int8_t* y,
                       const float* sy, void* out, hipStream_t st);

}  // namespace rece
