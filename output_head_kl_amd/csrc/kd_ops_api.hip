// C-ABI front end of the operators beside the loss (declared in include/kdkl.h): host-side
// argument checks before any HIP call, then the launches.  No call here synchronises,
// allocates device memory or copies, so each can be recorded into a HIP graph.
#include "kd_ops.h"
#include "kdkl.h"

#include <algorithm>
#include <new>
#include <vector>

namespace {

using kd::set_error;

inline int64_t rup(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline bool mis(const void *p, uintptr_t a) { return p && ((uintptr_t)p % a) != 0; }

#define LAUNCH(cls, expr)                                                              \
  do {                                                                                 \
    kd::prof_begin(cls, stream);                                                       \
    hipError_t e_ = (expr);                                                            \
    kd::prof_end(cls, stream);                                                         \
    if (e_ != hipSuccess)                                                              \
      return set_error(KD_E_HIP, "launch %s failed: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

int check_logits(const void *logits, int32_t dtype, int64_t ld, const void *tokens,
                 int32_t token_bits, int64_t N, int64_t V) {
  if (dtype != KD_F32 && dtype != KD_BF16) return set_error(KD_E_ARG, "dtype %d unknown", dtype);
  if (token_bits != 32 && token_bits != 64)
    return set_error(KD_E_ARG, "token_bits = %d: tokens are 32- or 64-bit integers", token_bits);
  if (N < 0 || V < 1) return set_error(KD_E_ARG, "need N >= 0 and V >= 1");
  if (N > 1 && ld < V) return set_error(KD_E_ARG, "ld = %lld is below V = %lld", (long long)ld, (long long)V);
  if (V >= ((int64_t)1 << 29) || N >= ((int64_t)1 << 24))
    return set_error(KD_E_UNSUPPORTED, "V must be below 2^29 and N below 2^24");
  if (N > 1 && ld > ((int64_t)1 << 36)) return set_error(KD_E_UNSUPPORTED, "ld must be at most 2^36");
  if (N > 0 && (!logits || !tokens)) return set_error(KD_E_ARG, "logits and tokens are required when N > 0");
  if (mis(logits, dtype == KD_BF16 ? 2 : 4)) return set_error(KD_E_ARG, "logits misaligned");
  if (mis(tokens, token_bits / 8)) return set_error(KD_E_ARG, "tokens misaligned");
  return KD_OK;
}

int check_tensors(const int64_t *numel, int32_t n) {
  if (n < 0) return set_error(KD_E_ARG, "n = %d < 0", n);
  if (n > 0 && !numel) return set_error(KD_E_ARG, "numel is required when n > 0");
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (numel[i] < 0) return set_error(KD_E_ARG, "numel[%d] = %lld < 0", i, (long long)numel[i]);
    if (numel[i] > ((int64_t)1 << 44) || (total += numel[i]) > ((int64_t)1 << 44))
      return set_error(KD_E_UNSUPPORTED, "more than 2^44 elements");
  }
  return KD_OK;
}

struct Span {
  uintptr_t lo, hi;
  int32_t i;
};

// Every element is written once, and only its own tensor's gradient may share its place.
int check_overlap(const void *const *grads, void *const *outs, const int64_t *numel,
                  const int32_t *dtypes, int32_t n) {
  std::vector<Span> w;
  w.reserve((size_t)n);
  auto bytes = [&](int32_t i) { return (uintptr_t)numel[i] * (dtypes[i] == KD_BF16 ? 2 : 4); };
  for (int32_t i = 0; i < n; ++i)
    if (numel[i] > 0) {
      const uintptr_t p = (uintptr_t)(outs ? outs[i] : grads[i]);
      w.push_back({p, p + bytes(i), i});
    }
  std::sort(w.begin(), w.end(), [](const Span &a, const Span &b) { return a.lo < b.lo; });
  for (size_t k = 1; k < w.size(); ++k)
    if (w[k].lo < w[k - 1].hi)
      return set_error(KD_E_ARG, "tensors %d and %d to be written share memory", w[k - 1].i, w[k].i);
  if (!outs) return KD_OK;
  for (int32_t i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t lo = (uintptr_t)grads[i], hi = lo + bytes(i);
    auto it = std::upper_bound(w.begin(), w.end(), lo,
                               [](uintptr_t x, const Span &s) { return x < s.hi; });
    for (; it != w.end() && it->lo < hi; ++it)
      if (!(it->i == i && it->lo == lo))
        return set_error(KD_E_ARG, "output %d shares memory with gradient %d", it->i, i);
  }
  return KD_OK;
}

}  // namespace

extern "C" {

int kd_token_logprobs_workspace_bytes(int64_t N, int64_t V, int32_t top, int32_t dtype,
                                      size_t *bytes_out) {
  set_error(KD_OK, nullptr);
  if (!bytes_out) return set_error(KD_E_ARG, "bytes_out is NULL");
  if (dtype != KD_F32 && dtype != KD_BF16) return set_error(KD_E_ARG, "dtype %d unknown", dtype);
  if (N < 0 || V < 1 || top < 0) return set_error(KD_E_ARG, "need N >= 0, V >= 1, top >= 0");
  if (top > kd::kLpMaxTop || V >= ((int64_t)1 << 29) || N >= ((int64_t)1 << 24))
    return set_error(KD_E_UNSUPPORTED, "top must be at most %d, V below 2^29 and N below 2^24",
                     kd::kLpMaxTop);
  *bytes_out = kd::lp_workspace(N, V, top, dtype);
  return KD_OK;
}

int kd_token_logprobs(const void *logits, int32_t dtype, int64_t ld, const void *tokens,
                      int32_t token_bits, int64_t N, int64_t V, int32_t top, float *logp,
                      float *entropy, float *row_lse, float *row_stats, int32_t *top_idx,
                      float *top_logp, int32_t *status, void *workspace, size_t workspace_bytes,
                      void *stream_v) {
  set_error(KD_OK, nullptr);
  int rc = check_logits(logits, dtype, ld, tokens, token_bits, N, V);
  if (rc != KD_OK) return rc;
  if (top < 0 || top > V) return set_error(KD_E_ARG, "top = %d outside [0, V = %lld]", top, (long long)V);
  if (top > kd::kLpMaxTop)
    return set_error(KD_E_UNSUPPORTED, "top = %d above %d", top, kd::kLpMaxTop);
  if (N > 0 && (!logp || !entropy || !row_lse))
    return set_error(KD_E_ARG, "logp, entropy and row_lse are required when N > 0");
  if (N > 0 && top > 0 && (!top_idx || !top_logp))
    return set_error(KD_E_ARG, "top_idx and top_logp are required when top > 0");
  if (mis(logp, 4) || mis(entropy, 4) || mis(row_lse, 4) || mis(top_idx, 4) || mis(top_logp, 4) ||
      mis(status, 4))
    return set_error(KD_E_ARG, "outputs must be 4-byte aligned");
  if (mis(row_stats, 8)) return set_error(KD_E_ARG, "row_stats must be 8-byte aligned");
  const size_t need = kd::lp_workspace(N, V, top, dtype);
  if (need > 0) {
    if (!workspace) return set_error(KD_E_WORKSPACE, "workspace is required (%zu bytes)", need);
    if (mis(workspace, 256)) return set_error(KD_E_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < need)
      return set_error(KD_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  }
  if (N == 0) return KD_OK;
  hipStream_t stream = (hipStream_t)stream_v;
  const kd::LpOut out{logp, entropy, row_lse, (float2 *)row_stats, top_idx, top_logp, status,
                      KD_E_INDEX};
  LAUNCH(kd::KC_LOGPROBS,
         kd::launch_token_logprobs(dtype, logits, ld, kd::Tokens{tokens, token_bits == 64}, N, V,
                                   top, out, workspace, stream));
  return KD_OK;
}

int kd_token_logprobs_bwd(const void *logits, int32_t dtype, int64_t ld, const void *tokens,
                          int32_t token_bits, int64_t N, int64_t V, const float *row_stats,
                          const float *entropy, const float *grad_logp, const float *grad_entropy,
                          const float *grad_lse, void *dlogits, int64_t ld_d, void *stream_v) {
  set_error(KD_OK, nullptr);
  int rc = check_logits(logits, dtype, ld, tokens, token_bits, N, V);
  if (rc != KD_OK) return rc;
  if (N > 1 && (ld_d < V || ld_d > ((int64_t)1 << 36)))
    return set_error(KD_E_ARG, "ld_d = %lld outside [V, 2^36]", (long long)ld_d);
  if (N > 0 && (!row_stats || !entropy || !dlogits))
    return set_error(KD_E_ARG, "row_stats, entropy and dlogits are required when N > 0");
  const int64_t es = dtype == KD_BF16 ? 2 : 4;
  if (mis(dlogits, es)) return set_error(KD_E_ARG, "dlogits misaligned");
  if (mis(row_stats, 8)) return set_error(KD_E_ARG, "row_stats must be 8-byte aligned");
  if (mis(entropy, 4) || mis(grad_logp, 4) || mis(grad_entropy, 4) || mis(grad_lse, 4))
    return set_error(KD_E_ARG, "float arguments must be 4-byte aligned");
  if (N == 0) return KD_OK;
  // in place only element for element: any other overlap would read what was written
  const uintptr_t a = (uintptr_t)logits, b = (uintptr_t)dlogits;
  const uintptr_t na = (uintptr_t)(((N - 1) * ld + V) * es), nb = (uintptr_t)(((N - 1) * ld_d + V) * es);
  if (a < b + nb && b < a + na && !(a == b && (N == 1 || ld == ld_d)))
    return set_error(KD_E_ARG, "dlogits overlaps logits and is not logits itself");
  // one workgroup per 8192 bf16 or 4096 fp32 elements of a row
  if (N * ((V * es + 16383) / 16384) > (int64_t)0x7FFFFFFF)
    return set_error(KD_E_UNSUPPORTED, "N x V is too large for one call");
  hipStream_t stream = (hipStream_t)stream_v;
  const kd::LpGrad g{(const float2 *)row_stats, entropy, grad_logp, grad_entropy, grad_lse};
  LAUNCH(kd::KC_LOGPROBS_BWD,
         kd::launch_token_logprobs_bwd(dtype, logits, ld, kd::Tokens{tokens, token_bits == 64}, N,
                                       V, g, dlogits, ld_d, stream));
  return KD_OK;
}

int kd_clip_grads_workspace_bytes(const int64_t *numel, int32_t n, size_t *bytes_out) {
  set_error(KD_OK, nullptr);
  if (!bytes_out) return set_error(KD_E_ARG, "bytes_out is NULL");
  int rc = check_tensors(numel, n);
  if (rc != KD_OK) return rc;
  *bytes_out = (size_t)rup((kd::clip_partials(numel, n) + 1) * 8, 256);
  return KD_OK;
}

int kd_clip_grads(const void *const *grads, void *const *outs, const int64_t *numel,
                  const int32_t *dtypes, int32_t n, float max_norm, float *norm, void *workspace,
                  size_t workspace_bytes, void *stream_v) {
  set_error(KD_OK, nullptr);
  int rc = check_tensors(numel, n);
  if (rc != KD_OK) return rc;
  if (!(max_norm >= 0.f)) return set_error(KD_E_ARG, "max_norm must be >= 0 (infinity: no clipping)");
  if (n > 0 && (!grads || !dtypes)) return set_error(KD_E_ARG, "grads and dtypes are required when n > 0");
  if (!norm || mis(norm, 4)) return set_error(KD_E_ARG, "norm is required, 4-byte aligned");
  for (int32_t i = 0; i < n; ++i) {
    if (dtypes[i] != KD_F32 && dtypes[i] != KD_BF16)
      return set_error(KD_E_ARG, "dtypes[%d] = %d unknown", i, dtypes[i]);
    if (numel[i] == 0) continue;
    const uintptr_t es = dtypes[i] == KD_BF16 ? 2 : 4;
    if (!grads[i] || (outs && !outs[i])) return set_error(KD_E_ARG, "tensor %d is NULL", i);
    if (mis(grads[i], es) || (outs && mis(outs[i], es)))
      return set_error(KD_E_ARG, "tensor %d is misaligned", i);
  }
  const bool scale = outs || max_norm < __builtin_huge_valf();
  if (scale) {
    try {
      rc = check_overlap(grads, outs, numel, dtypes, n);
    } catch (const std::bad_alloc &) {
      return set_error(KD_E_ARG, "out of host memory for %d tensors", n);
    }
    if (rc != KD_OK) return rc;
  }
  const size_t need = (size_t)rup((kd::clip_partials(numel, n) + 1) * 8, 256);
  if (!workspace) return set_error(KD_E_WORKSPACE, "workspace is required (%zu bytes)", need);
  if (mis(workspace, 256)) return set_error(KD_E_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < need)
    return set_error(KD_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  hipStream_t stream = (hipStream_t)stream_v;
  LAUNCH(kd::KC_CLIP, kd::launch_clip_grads(grads, outs, numel, dtypes, n, scale, max_norm, norm,
                                            (double *)workspace, stream));
  return KD_OK;
}

}  // extern "C"
