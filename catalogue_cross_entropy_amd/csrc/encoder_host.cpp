// C entry points of the sequence encoder's operators (attention, residual norm) and of 8-bit scoring:
// argument checks, then the launchers of k_attention.hip, k_norm.hip and k_int8.hip.  Nothing here allocates
// or waits.
#include <hip/hip_runtime.h>

#include <cmath>

#include "rece_ops.h"

using namespace rece;

namespace {

constexpr int64_t I32_MAX = ((int64_t)1 << 31) - 1;

rece_status invalid(const char* msg) { return set_last_error(RECE_ERR_INVALID_ARGUMENT, msg); }
rece_status unsupported(const char* msg) { return set_last_error(RECE_ERR_UNSUPPORTED, msg); }
rece_status too_small(const char* msg) { return set_last_error(RECE_ERR_WORKSPACE_TOO_SMALL, msg); }

rece_status hip_status(hipError_t e) {
  return e == hipSuccess ? RECE_OK : set_last_error(RECE_ERR_HIP, hipGetErrorString(e));
}

template <class... P>
bool misaligned(unsigned a, P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & (a - 1)) != 0;
}
template <class... P>
bool missing(P... p) {
  return (!p || ...);
}

bool bad_dtype(int32_t t) { return t != RECE_F32 && t != RECE_BF16; }

// offsets within a tile of up to 64 rows stay below 2^31 bytes
bool bad_stride(int64_t stride, int64_t row) { return stride < row || stride % 8 != 0 || stride > (1 << 23); }

rece_status check_attention(const rece_attention_config* c) {
  if (!c) return invalid("config is NULL");
  if (c->n < 0 || c->n_seq < 1) return invalid("n must be >= 0 and n_seq >= 1");
  if (c->n > I32_MAX || c->n_seq > I32_MAX - 1) return unsupported("n and n_seq must fit in int32");
  if (bad_dtype(c->dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (c->d < 1 || c->heads < 1 || c->kv_heads < 1) return invalid("d, heads and kv_heads must be >= 1");
  if (c->d % 8 != 0 || c->d > 128) return unsupported("d must be a multiple of 8, at most 128");
  if (c->heads % c->kv_heads != 0) return invalid("heads must be a multiple of kv_heads");
  if (c->heads > 1024) return unsupported("heads must be at most 1024");
  if (!(c->scale > 0.0f) || !std::isfinite(c->scale)) return invalid("scale must be positive and finite");
  if (bad_stride(c->q_stride, (int64_t)c->heads * c->d) || bad_stride(c->k_stride, (int64_t)c->kv_heads * c->d) ||
      bad_stride(c->v_stride, (int64_t)c->kv_heads * c->d))
    return invalid("strides must be multiples of 8, at least a row's elements, at most 2^23");
  if (c->n_bounds < 0 || c->n_bounds > RECE_MAX_BOUNDS) return invalid("n_bounds must be in [0, RECE_MAX_BOUNDS]");
  for (int t = 0; t < c->n_bounds; ++t)
    if (c->bounds[t] < 1 || c->bounds[t] > RECE_MAX_DISTANCE || (t > 0 && c->bounds[t] <= c->bounds[t - 1]))
      return invalid("bounds must be increasing distances in [1, RECE_MAX_DISTANCE]");
  return RECE_OK;
}

// sizes of a packed call: a grid holds less than 2^32 lanes, 2^24 workgroups of 256
rece_status check_packed(const rece_attention_config* c) {
  const rece_status v = check_attention(c);
  if (v != RECE_OK) return v;
  if ((c->n / 32 + c->n_seq) * c->heads > (1 << 24) - 1024) return unsupported("(n / 32 + n_seq) * heads must be below 2^24 - 1024");
  return RECE_OK;
}

rece_status check_last(const rece_attention_config* c, int64_t max_len) {
  const rece_status v = check_attention(c);
  if (v != RECE_OK) return v;
  if (max_len < 1) return invalid("max_len must be >= 1");
  if (c->heads / c->kv_heads > 32) return unsupported("heads / kv_heads must be at most 32");
  // (a grid of n_seq * kv_heads workgroups of 256 lanes, and of n_seq * heads joins of 1,024 lanes, below 2^32 lanes)
  if (c->n_seq * c->heads >= 1 << 22) return unsupported("n_seq * heads must be below 2^22");
  return RECE_OK;
}

rece_status check_norm(int64_t n, int32_t d) {
  if (n < 0 || d < 1) return invalid("n must be >= 0 and d >= 1");
  if (n > I32_MAX) return unsupported("n must fit in int32");
  if (d % 8 != 0 || d > 8192) return unsupported("d must be a multiple of 8, at most 8192");
  return RECE_OK;
}

}  // namespace

extern "C" {

rece_status rece_attention_workspace_bytes(const rece_attention_config* cfg, size_t* bytes) {
  const rece_status v = check_packed(cfg);
  if (v != RECE_OK) return v;
  if (!bytes) return invalid("bytes is NULL");
  *bytes = attention_workspace_bytes(*cfg);
  return RECE_OK;
}

rece_status rece_attention_forward(const rece_attention_config* cfg, void* stream, const void* q, const void* k,
                                   const void* v, const int32_t* offsets, const float* bias, void* workspace,
                                   size_t workspace_bytes, void* out) {
  const rece_status r = check_packed(cfg);
  if (r != RECE_OK) return r;
  if (cfg->n == 0) return RECE_OK;
  if (missing(q, k, v, offsets, out)) return invalid("NULL pointer argument");
  if (misaligned(16, q, k, v, out, workspace) || misaligned(4, offsets, bias))
    return invalid("q, k, v, out and workspace must be 16-byte aligned, offsets and bias 4-byte aligned");
  if (workspace && workspace_bytes < attention_workspace_bytes(*cfg))
    return too_small("workspace smaller than rece_attention_workspace_bytes");
  return hip_status(attention_forward(*cfg, q, k, v, offsets, bias, workspace, out, static_cast<hipStream_t>(stream)));
}

rece_status rece_attention_backward(const rece_attention_config* cfg, void* stream, const void* q, const void* k,
                                    const void* v, const int32_t* offsets, const float* bias, const void* out,
                                    void* workspace, size_t workspace_bytes, const void* dout, int64_t dq_stride,
                                    int64_t dk_stride, int64_t dv_stride, void* dq, void* dk, void* dv, float* dbias) {
  const rece_status r = check_packed(cfg);
  if (r != RECE_OK) return r;
  if (bad_stride(dq_stride, (int64_t)cfg->heads * cfg->d) || bad_stride(dk_stride, (int64_t)cfg->kv_heads * cfg->d) ||
      bad_stride(dv_stride, (int64_t)cfg->kv_heads * cfg->d))
    return invalid("strides must be multiples of 8, at least a row's elements, at most 2^23");
  if (!bias != !dbias) return invalid("dbias goes with bias");
  if (misaligned(4, offsets, bias, dbias)) return invalid("offsets, bias and dbias must be 4-byte aligned");
  if (cfg->n > 0) {
    if (missing(q, k, v, offsets, out, workspace, dout, dq, dk, dv)) return invalid("NULL pointer argument");
    if (misaligned(16, q, k, v, out, workspace, dout, dq, dk, dv))
      return invalid("q, k, v, out, workspace, dout, dq, dk and dv must be 16-byte aligned");
    if (workspace_bytes < attention_workspace_bytes(*cfg))
      return too_small("workspace smaller than rece_attention_workspace_bytes");
  }
  return hip_status(attention_backward(*cfg, q, k, v, offsets, bias, out, workspace, dout, dq, dk, dv, dbias,
                                       {dq_stride, dk_stride, dv_stride}, static_cast<hipStream_t>(stream)));
}

rece_status rece_last_attention_workspace_bytes(const rece_attention_config* cfg, int64_t max_len, size_t* bytes) {
  const rece_status v = check_last(cfg, max_len);
  if (v != RECE_OK) return v;
  if (!bytes) return invalid("bytes is NULL");
  *bytes = last_attention_workspace_bytes(*cfg, max_len);
  return RECE_OK;
}

rece_status rece_last_attention(const rece_attention_config* cfg, void* stream, int64_t max_len, const void* q,
                                const void* k, const void* v, const int32_t* begin, const int32_t* length,
                                const float* bias, void* workspace, size_t workspace_bytes, void* out) {
  const rece_status r = check_last(cfg, max_len);
  if (r != RECE_OK) return r;
  if (missing(q, begin, length, out) || (cfg->n > 0 && missing(k, v))) return invalid("NULL pointer argument");
  if (misaligned(16, q, k, v, out, workspace) || misaligned(4, begin, length, bias))
    return invalid("q, k, v, out and workspace must be 16-byte aligned, begin, length and bias 4-byte aligned");
  const size_t need = last_attention_workspace_bytes(*cfg, max_len);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return too_small("workspace smaller than rece_last_attention_workspace_bytes");
  return hip_status(last_attention(*cfg, max_len, q, k, v, begin, length, bias, workspace, out,
                                   static_cast<hipStream_t>(stream)));
}

rece_status rece_norm_workspace_bytes(int64_t n, int32_t d, size_t* bytes) {
  const rece_status v = check_norm(n, d);
  if (v != RECE_OK) return v;
  if (!bytes) return invalid("bytes is NULL");
  *bytes = norm_workspace_bytes(n, d);
  return RECE_OK;
}

rece_status rece_norm_forward(void* stream, int64_t n, int32_t d, int32_t dtype, float eps, const void* x,
                              const void* residual, const float* weight, void* h, void* y, float* rstd) {
  const rece_status v = check_norm(n, d);
  if (v != RECE_OK) return v;
  if (bad_dtype(dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return invalid("eps must be finite and >= 0");
  if (n == 0) return RECE_OK;
  if (missing(x, weight, y)) return invalid("NULL pointer argument");
  if (misaligned(16, x, residual, weight, h, y) || misaligned(4, rstd))
    return invalid("x, residual, weight, h and y must be 16-byte aligned, rstd 4-byte aligned");
  return hip_status(norm_forward(dtype == RECE_BF16, n, d, eps, x, residual, weight, h, y, rstd,
                                 static_cast<hipStream_t>(stream)));
}

rece_status rece_norm_forward_int8(void* stream, int64_t n, int32_t d, int32_t dtype, float eps, const void* x,
                                   const void* residual, const float* weight, void* h, int8_t* y8, float* scale) {
  const rece_status v = check_norm(n, d);
  if (v != RECE_OK) return v;
  if (bad_dtype(dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return invalid("eps must be finite and >= 0");
  if (n == 0) return RECE_OK;
  if (missing(x, weight, y8, scale)) return invalid("NULL pointer argument");
  if (misaligned(16, x, residual, weight, h, y8) || misaligned(4, scale))
    return invalid("x, residual, weight, h and y8 must be 16-byte aligned, scale 4-byte aligned");
  return hip_status(norm_forward_int8(dtype == RECE_BF16, n, d, eps, x, residual, weight, h, y8, scale,
                                      static_cast<hipStream_t>(stream)));
}

rece_status rece_norm_backward(void* stream, int64_t n, int32_t d, int32_t dtype, const void* dy, const void* h,
                               const void* dh, const float* weight, const float* rstd, void* workspace,
                               size_t workspace_bytes, void* dx, float* dweight) {
  const rece_status v = check_norm(n, d);
  if (v != RECE_OK) return v;
  if (bad_dtype(dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (!dweight || (n > 0 && missing(dy, h, weight, rstd, workspace, dx))) return invalid("NULL pointer argument");
  if (misaligned(16, dy, h, dh, weight, workspace, dx) || misaligned(4, rstd, dweight))
    return invalid("dy, h, dh, weight, workspace and dx must be 16-byte aligned, rstd and dweight 4-byte aligned");
  if (workspace_bytes < norm_workspace_bytes(n, d)) return too_small("workspace smaller than rece_norm_workspace_bytes");
  return hip_status(norm_backward(dtype == RECE_BF16, n, d, dy, h, dh, weight, rstd, workspace, dx, dweight,
                                  static_cast<hipStream_t>(stream)));
}

rece_status rece_quantize_rows(void* stream, int64_t n, int32_t d, int32_t dtype, const void* x, int8_t* x8,
                               float* scale) {
  const rece_status v = check_norm(n, d);
  if (v != RECE_OK) return v;
  if (bad_dtype(dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (n == 0) return RECE_OK;
  if (missing(x, x8, scale)) return invalid("NULL pointer argument");
  if (misaligned(16, x, x8) || misaligned(4, scale)) return invalid("x and x8 must be 16-byte aligned, scale 4-byte aligned");
  return hip_status(quantize_rows(dtype == RECE_BF16, n, d, x, x8, scale, static_cast<hipStream_t>(stream)));
}

rece_status rece_int8_scores(void* stream, int64_t s, int64_t C, int32_t d, int32_t dtype, const int8_t* x8,
                             const float* sx, const int8_t* y8, const float* sy, void* out) {
  if (s < 0 || C < 1 || d < 1) return invalid("s must be >= 0, C and d >= 1");
  if (s > I32_MAX || C > I32_MAX) return unsupported("s and C must fit in int32");
  if (d > 256 && int8_tiles(s, C) >= 1 << 24) return unsupported("more than 2^24 tiles of 128 x 128 scores with d beyond 256");
  if (d % 16 != 0 || d > 8192) return unsupported("d must be a multiple of 16, at most 8192");
  if (bad_dtype(dtype)) return unsupported("dtype must be RECE_F32 or RECE_BF16");
  if (s == 0) return RECE_OK;
  if (missing(x8, sx, y8, sy, out)) return invalid("NULL pointer argument");
  if (misaligned(16, x8, y8) || misaligned(dtype == RECE_BF16 ? 2 : 4, out) || misaligned(4, sx, sy))
    return invalid("x8 and y8 must be 16-byte aligned, sx, sy and out aligned to their elements");
  return hip_status(int8_scores(dtype == RECE_BF16, s, C, d, x8, sx, y8, sy, out, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
