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

int check_head(const void *h, const void *W, int32_t dtype, const void *tokens, int32_t token_bits,
               int64_t N, int64_t d, int64_t V, int64_t chunk, bool pointers) {
  if (dtype != KD_F32 && dtype != KD_BF16) return set_error(KD_E_ARG, "dtype %d unknown", dtype);
  if (N < 0 || d < 1 || V < 1) return set_error(KD_E_ARG, "need N >= 0, d >= 1, V >= 1");
  if (chunk < 1) return set_error(KD_E_ARG, "chunk = %lld < 1", (long long)chunk);
  if (d % 8 != 0)
    return set_error(KD_E_UNSUPPORTED, "d = %lld is not a multiple of 8", (long long)d);
  if (d > (1 << 20) || V > ((int64_t)1 << 24) || N > ((int64_t)1 << 40))
    return set_error(KD_E_UNSUPPORTED, "d must be at most 2^20, V 2^24 and N 2^40");
  if ((chunk < N ? chunk : N) > ((int64_t)1 << 22))
    return set_error(KD_E_UNSUPPORTED, "min(chunk, N) must be at most 2^22 rows");
  // a launch has fewer than 2^32 threads
  if ((chunk < N ? chunk : N) * V > ((int64_t)1 << 38))
    return set_error(KD_E_UNSUPPORTED, "min(chunk, N) x V must be at most 2^38");
  if (!pointers) return KD_OK;
  if (token_bits != 32 && token_bits != 64)
    return set_error(KD_E_ARG, "token_bits = %d: tokens are 32- or 64-bit integers", token_bits);
  if (!W) return set_error(KD_E_ARG, "W is required");
  if (N > 0 && (!h || !tokens)) return set_error(KD_E_ARG, "h and tokens are required when N > 0");
  if (mis(h, 16) || mis(W, 16)) return set_error(KD_E_ARG, "h and W must be 16-byte aligned");
  if (mis(tokens, token_bits / 8)) return set_error(KD_E_ARG, "tokens misaligned");
  return KD_OK;
}

inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

int check_workspace(const void *workspace, size_t bytes, size_t need) {
  if (!workspace) return set_error(KD_E_WORKSPACE, "workspace is required (%zu bytes)", need);
  if (mis(workspace, 256)) return set_error(KD_E_ARG, "workspace must be 256-byte aligned");
  if (bytes < need)
    return set_error(KD_E_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
  return KD_OK;
}

// Forward workspace: the partials of one chunk and its given tokens' logits.
struct HeadFwd {
  int64_t C, C_alloc, n_lse;
  bool few;  // few tokens in all: one pass that streams W, whatever the chunk
  size_t off_t, off_zt, total;
};
HeadFwd head_fwd_layout(int64_t N, int64_t V, int64_t chunk, int dtype) {
  HeadFwd L;
  L.C = chunk < N ? chunk : (N > 0 ? N : 1);
  L.C_alloc = rup(L.C, 64);
  const int64_t wr = kd::head_part_rows(dtype, L.C, V);
  L.few = N <= kd::kHeadFewTokens;
  if (L.few) L.C = L.C_alloc = N > 0 ? N : 1;
  L.n_lse = L.few ? kd::head_few_partials(L.C, V) : (V + wr - 1) / wr;
  L.off_t = (size_t)rup(L.n_lse * L.C_alloc * 8, 256);
  L.off_zt = L.off_t + (size_t)rup(L.n_lse * L.C_alloc * 4, 256);
  L.total = L.off_zt + (size_t)rup(L.C_alloc * 4, 256);
  return L;
}

// Backward workspace.  The dW sum runs over groups of chunks; with more than one group and
// dW not float32 the sum of the earlier ones is kept in float32 here.
struct HeadBwd {
  int64_t C, C_alloc, V_pad, d_pad, nchunks, group, k_split;
  int nsplit;
  bool few; // bf16, few tokens in all: one pass over W gives dz and dW
  bool wt;  // bf16: the dh product reads a k-contiguous copy of W
  size_t off_coef, off_dz, off_dhpart, off_wt, off_dzt, off_ht, off_acc, total;
};
HeadBwd head_bwd_layout(int64_t N, int64_t d, int64_t V, int64_t chunk, int dtype, int dw_dtype,
                        bool want_dh, bool want_dw, int64_t group) {
  HeadBwd L;
  const bool bf16 = dtype == KD_BF16;
  const int64_t es = bf16 ? 2 : 4, n = N > 0 ? N : 1;
  L.few = bf16 && n <= kd::kHeadFewTokens;
  L.C = chunk < n && !L.few ? chunk : n;
  L.C_alloc = rup(L.C, kd::kTile);
  L.V_pad = rup(V, bf16 && !L.few ? 3 * kd::kTile : kd::kTile);
  L.d_pad = rup(d, kd::kTile);
  L.nchunks = (n + L.C - 1) / L.C;
  L.group = !bf16 || group < 1 ? 1 : group < L.nchunks ? group : L.nchunks;
  L.wt = bf16 && !L.few && kd::head_wt(n, L.C_alloc, d, L.V_pad);
  if (L.few) L.nsplit = kd::head_few_dh_splits(d, V);
  else kd::head_dh_splits(dtype, L.wt, L.C_alloc, d, L.V_pad, &L.nsplit, &L.k_split);
  const int64_t tok = kd::head_few_tokens(n);
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = off;
    off += (size_t)rup(bytes, 256);
    return o;
  };
  L.off_coef = take(L.few ? 0 : 5 * L.C_alloc * 4);
  L.off_dz = take(!L.few ? L.C_alloc * L.V_pad * es : want_dh ? 2 * tok * L.V_pad * 2 : 0);
  L.off_dhpart =
      take(!want_dh ? 0 : L.nsplit * 4 * (L.few ? tok * rup(d, 128) : L.C_alloc * L.d_pad));
  L.off_wt = take(want_dh && L.wt ? L.V_pad * d * 2 : 0);
  L.off_dzt = take(want_dw && bf16 && !L.few ? L.group * L.C_alloc * L.V_pad * 2 : 0);
  L.off_ht = take(want_dw && bf16 ? L.group * L.C_alloc * d * 2 : 0);
  L.off_acc = take(want_dw && dw_dtype != KD_F32 && L.group < L.nchunks ? V * d * 4 : 0);
  L.total = off;
  return L;
}

// Chunks per group of at most `tokens` tokens (at most kDwGroupTokens, as in the loss).
int64_t group_chunks(int64_t tokens, int64_t N, int64_t chunk) {
  const int64_t n = N > 0 ? N : 1, C = rup(chunk < n ? chunk : n, kd::kTile);
  const int64_t t = tokens < kd::kDwGroupTokens ? tokens : kd::kDwGroupTokens;
  return t / C < 1 ? 1 : t / C;
}

kd::Tokens tokens_at(const void *tokens, int32_t token_bits, int64_t c0) {
  return kd::Tokens{(const char *)tokens + c0 * (token_bits / 8), token_bits == 64};
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
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != KD_OK) return rc;
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
  // one workgroup of 256 per 8192 bf16 or 4096 fp32 elements of a row: fewer than 2^32 threads
  if (N * ((V * es + 16383) / 16384) >= ((int64_t)1 << 24))
    return set_error(KD_E_UNSUPPORTED, "N x V is too large for one call");
  hipStream_t stream = (hipStream_t)stream_v;
  const kd::LpGrad g{(const float2 *)row_stats, entropy, grad_logp, grad_entropy, grad_lse};
  LAUNCH(kd::KC_LOGPROBS_BWD,
         kd::launch_token_logprobs_bwd(dtype, logits, ld, kd::Tokens{tokens, token_bits == 64}, N,
                                       V, g, dlogits, ld_d, stream));
  return KD_OK;
}

int kd_head_logprobs_workspace_bytes(int64_t N, int64_t d, int64_t V, int64_t chunk,
                                     int32_t dtype, size_t *bytes_out) {
  set_error(KD_OK, nullptr);
  if (!bytes_out) return set_error(KD_E_ARG, "bytes_out is NULL");
  int rc = check_head(nullptr, nullptr, dtype, nullptr, 0, N, d, V, chunk, false);
  if (rc != KD_OK) return rc;
  *bytes_out = head_fwd_layout(N, V, chunk, dtype).total;
  return KD_OK;
}

int kd_head_logprobs(const void *h, const void *W, int32_t dtype, const void *tokens,
                     int32_t token_bits, int64_t N, int64_t d, int64_t V, int64_t chunk,
                     float *logp, float *entropy, float *row_lse, float *row_stats,
                     int32_t *status, void *workspace, size_t workspace_bytes, void *stream_v) {
  set_error(KD_OK, nullptr);
  int rc = check_head(h, W, dtype, tokens, token_bits, N, d, V, chunk, true);
  if (rc != KD_OK) return rc;
  if (N > 0 && (!logp || !entropy || !row_lse))
    return set_error(KD_E_ARG, "logp, entropy and row_lse are required when N > 0");
  if (mis(logp, 4) || mis(entropy, 4) || mis(row_lse, 4) || mis(status, 4))
    return set_error(KD_E_ARG, "outputs must be 4-byte aligned");
  if (mis(row_stats, 8)) return set_error(KD_E_ARG, "row_stats must be 8-byte aligned");
  const HeadFwd L = head_fwd_layout(N, V, chunk, dtype);
  rc = check_workspace(workspace, workspace_bytes, L.total);
  if (rc != KD_OK) return rc;
  hipStream_t stream = (hipStream_t)stream_v;
  float2 *part = (float2 *)workspace;
  float *part_t = (float *)((char *)workspace + L.off_t);
  float *zt = (float *)((char *)workspace + L.off_zt);
  const int64_t es = dtype == KD_BF16 ? 2 : 4;
  for (int64_t c0 = 0; c0 < N; c0 += L.C) {
    const int64_t rows = N - c0 < L.C ? N - c0 : L.C;
    const char *h_c = (const char *)h + c0 * d * es;
    const kd::Tokens tok = tokens_at(tokens, token_bits, c0);
    LAUNCH(kd::KC_FWD_GEMM,
           L.few ? kd::launch_head_few(dtype, W, h_c, rows, d, V, tok, part, part_t, zt, stream)
                 : kd::launch_head_fwd(dtype, W, h_c, rows, d, V, tok, part, part_t, L.C_alloc,
                                       L.C, zt, stream));
    const kd::LpOut out{logp + c0, entropy + c0, row_lse + c0,
                        row_stats ? (float2 *)row_stats + c0 : nullptr, nullptr, nullptr, status,
                        KD_E_INDEX};
    LAUNCH(kd::KC_LOGPROBS, kd::launch_head_join(L.few, part, part_t, L.n_lse, L.C_alloc, rows, V,
                                                 zt, tok, out, stream));
  }
  return KD_OK;
}

int kd_head_logprobs_bwd_workspace_bytes(int64_t N, int64_t d, int64_t V, int64_t chunk,
                                         int32_t dtype, int32_t dw_dtype,
                                         int64_t dw_group_tokens, size_t *bytes_out) {
  set_error(KD_OK, nullptr);
  if (!bytes_out) return set_error(KD_E_ARG, "bytes_out is NULL");
  int rc = check_head(nullptr, nullptr, dtype, nullptr, 0, N, d, V, chunk, false);
  if (rc != KD_OK) return rc;
  if (dw_dtype != KD_F32 && dw_dtype != dtype)
    return set_error(KD_E_ARG, "dw_dtype is KD_F32 or dtype");
  if (dw_group_tokens < 0) return set_error(KD_E_ARG, "dw_group_tokens is negative");
  *bytes_out = head_bwd_layout(N, d, V, chunk, dtype, dw_dtype, true, true,
                               group_chunks(dw_group_tokens, N, chunk)).total;
  return KD_OK;
}

int kd_head_logprobs_bwd(const void *h, const void *W, int32_t dtype, const void *tokens,
                         int32_t token_bits, int64_t N, int64_t d, int64_t V, int64_t chunk,
                         const float *row_stats, const float *entropy, const float *grad_logp,
                         const float *grad_entropy, const float *grad_lse, void *dh, void *dW,
                         int32_t dw_dtype, void *workspace, size_t workspace_bytes,
                         void *stream_v) {
  set_error(KD_OK, nullptr);
  int rc = check_head(h, W, dtype, tokens, token_bits, N, d, V, chunk, true);
  if (rc != KD_OK) return rc;
  if (!dh && !dW) return set_error(KD_E_ARG, "neither dh nor dW is wanted");
  if (dw_dtype != KD_F32 && dw_dtype != dtype)
    return set_error(KD_E_ARG, "dw_dtype is KD_F32 or dtype");
  if (N > 0 && (!row_stats || !entropy))
    return set_error(KD_E_ARG, "row_stats and entropy are required when N > 0");
  if (mis(row_stats, 8)) return set_error(KD_E_ARG, "row_stats must be 8-byte aligned");
  if (mis(entropy, 4) || mis(grad_logp, 4) || mis(grad_entropy, 4) || mis(grad_lse, 4))
    return set_error(KD_E_ARG, "float arguments must be 4-byte aligned");
  if (mis(dh, 16) || mis(dW, 16)) return set_error(KD_E_ARG, "dh and dW must be 16-byte aligned");
  // the dW group is the largest (up to kDwGroupTokens tokens) that fits
  HeadBwd L;
  for (int64_t g = group_chunks(kd::kDwGroupTokens, N, chunk); g >= 1; --g) {
    L = head_bwd_layout(N, d, V, chunk, dtype, dw_dtype, dh != nullptr, dW != nullptr, g);
    if (workspace_bytes >= L.total) break;
  }
  rc = check_workspace(workspace, workspace_bytes, L.total);
  if (rc != KD_OK) return rc;
  hipStream_t stream = (hipStream_t)stream_v;
  const bool bf16 = dtype == KD_BF16;
  // a chunk's results are written before the next one reads h and W
  const int64_t nh = N * d * (bf16 ? 2 : 4), nW = V * d * (bf16 ? 2 : 4);
  const int64_t nG = V * d * (dw_dtype == KD_F32 ? 4 : 2);
  if (overlap(dh, nh, h, nh) || overlap(dh, nh, W, nW) || overlap(dW, nG, h, nh) ||
      overlap(dW, nG, W, nW) || overlap(dh, nh, dW, nG))
    return set_error(KD_E_ARG, "dh and dW may not share memory with h, W or each other");
  const int64_t es = bf16 ? 2 : 4, tst_dz = L.V_pad * 256, tst_h = d * 256;
  if (N == 0) {
    if (dW)
      LAUNCH(kd::KC_MISC,
             kd::launch_fill_zero(dW, (size_t)V * d * (dw_dtype == KD_F32 ? 4 : 2), stream));
    return KD_OK;
  }
  char *ws = (char *)workspace;
  float *coef = (float *)(ws + L.off_coef);
  const kd::HeadCoef k{coef, coef + L.C_alloc, coef + 2 * L.C_alloc, coef + 3 * L.C_alloc,
                       (int *)(coef + 4 * L.C_alloc)};
  void *dz = ws + L.off_dz, *WT = L.wt ? ws + L.off_wt : nullptr;
  float *dhpart = (float *)(ws + L.off_dhpart);
  if (dh && WT)
    LAUNCH(kd::KC_TRANSPOSE, kd::launch_transpose_w(W, V, d, L.V_pad, WT, stream));
  if (L.few) {
    const kd::LpGrad g{(const float2 *)row_stats, entropy, grad_logp, grad_entropy, grad_lse};
    void *ht = ws + L.off_ht;
    if (dW) LAUNCH(kd::KC_TRANSPOSE, kd::launch_transpose_h(h, N, d, L.C_alloc, ht, tst_h, stream));
    LAUNCH(kd::KC_BWD_GEMM,
           kd::launch_head_few_bwd(W, h, ht, N, d, V, L.V_pad, tokens_at(tokens, token_bits, 0), g,
                                   dh ? dz : nullptr, dW, dw_dtype, stream));
    if (dh)
      LAUNCH(kd::KC_DH_GEMM, kd::launch_head_few_dh(W, dz, N, d, V, L.V_pad, L.nsplit, dhpart, dh,
                                                    stream));
    return KD_OK;
  }
  int64_t chunk_i = 0;
  float *sum = nullptr;  // the earlier groups' sum
  for (int64_t c0 = 0; c0 < N; c0 += L.C, ++chunk_i) {
    const int64_t rows = N - c0 < L.C ? N - c0 : L.C;
    const char *h_c = (const char *)h + c0 * d * es;
    const kd::LpGrad g{(const float2 *)row_stats + c0, entropy + c0,
                       grad_logp ? grad_logp + c0 : nullptr,
                       grad_entropy ? grad_entropy + c0 : nullptr,
                       grad_lse ? grad_lse + c0 : nullptr};
    LAUNCH(kd::KC_LOGPROBS_BWD,
           kd::launch_head_coef(tokens_at(tokens, token_bits, c0), g, rows, V, k, stream));
    const int64_t slot = chunk_i % L.group;
    void *dzt_c = bf16 && dW ? ws + L.off_dzt + (size_t)slot * L.C_alloc * L.V_pad * 2 : nullptr;
    LAUNCH(kd::KC_BWD_GEMM, kd::launch_head_dz(dtype, W, h_c, rows, d, V, k, dz, dzt_c, tst_dz,
                                               L.V_pad, L.C_alloc, stream));
    if (dh) {
      LAUNCH(kd::KC_DH_GEMM, kd::launch_head_dh(dtype, dz, W, WT, rows, d, V, L.V_pad, L.nsplit,
                                                L.k_split, dhpart, L.d_pad, L.C_alloc, stream));
      LAUNCH(kd::KC_DH_REDUCE, kd::launch_dh_reduce(dtype, dhpart, L.nsplit, L.C_alloc, L.d_pad,
                                                    rows, d, (char *)dh + c0 * d * es, stream));
    }
    if (!dW) continue;
    void *ht = bf16 ? ws + L.off_ht : nullptr;
    if (bf16)
      LAUNCH(kd::KC_TRANSPOSE,
             kd::launch_transpose_h(h_c, rows, d, L.C_alloc,
                                    (char *)ht + (size_t)slot * L.C_alloc * d * 2, tst_h, stream));
    const bool last = c0 + rows >= N;
    if (slot == L.group - 1 || last) {
      // every earlier chunk of the group is whole: its columns past C are zero
      const int64_t kk = slot * L.C_alloc + rows;
      const int out = last ? dw_dtype : (int)KD_F32;
      void *to = last || dw_dtype == KD_F32 ? dW : (void *)(ws + L.off_acc);
      LAUNCH(kd::KC_DW_GEMM,
             kd::launch_head_dw(dtype, out, dz, bf16 ? ws + L.off_dzt : nullptr, h_c, ht, kk, d, V,
                                L.V_pad, L.C_alloc, sum, to, stream));
      sum = (float *)to;
    }
  }
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
  rc = check_workspace(workspace, workspace_bytes,
                       (size_t)rup((kd::clip_partials(numel, n) + 1) * 8, 256));
  if (rc != KD_OK) return rc;
  hipStream_t stream = (hipStream_t)stream_v;
  LAUNCH(kd::KC_CLIP, kd::launch_clip_grads(grads, outs, numel, dtypes, n, scale, max_norm, norm,
                                            (double *)workspace, stream));
  return KD_OK;
}

}  // extern "C"
