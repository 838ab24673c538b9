// Internal interface of the operators beside the loss: log probabilities of given tokens
// (from logits and from hidden states) with their gradients, and gradient clipping.
#pragma once

#include "kd_internal.h"

namespace kd {

// ln(x) and 2^x of the hardware work in base 2.
constexpr float kOpLog2e = 1.4426950408889634f;
constexpr double kOpLn2d = 0.6931471805599453;
// Lower bound put on ln p where it multiplies p: p is 0 below about -104, and 0 * -inf is NaN.
constexpr float kOpLowest = -1.0e4f;

// The given tokens: int32 or int64, negative = the row has none.
struct Tokens {
  const void *ptr;
  int wide;  // 1: int64
  __device__ __forceinline__ long long at(long long n) const {
    return wide ? ((const long long *)ptr)[n] : (long long)((const int *)ptr)[n];
  }
};

// Per-row results.  stats[n] = (max, ln sum exp(z - max)), the state the gradients read
// (kept apart: their sum would lose digits of ln p where the maximum is large).
struct LpOut {
  float *logp, *entropy, *lse;
  float2 *stats;       // may be null
  int32_t *top_idx;    // [N][top], null when top == 0
  float *top_logp;
  int32_t *status;     // may be null; set to bad_code, never cleared
  int bad_code;
};

// ln S of a row with maximum m and S = sum exp(z - m): NaN for a bad row (a NaN or +inf logit),
// -inf for an empty one (no finite logit, S = 0).  S >= 1 holds the maximum's own term 1: ln S
// keeps its digits there through ln(1 + x).
__device__ __forceinline__ float lp_log(float m, double S) {
  if (!(S >= 0.0) || !(m < INFINITY)) return __uint_as_float(0x7FC00000u);
  if (S == 0.0) return -INFINITY;
  return S < 2.0 ? log1pf((float)(S - 1.0)) : logf((float)S);
}

// Writes a row's results from m, S, lnS = lp_log(m, S), T = sum exp(z - m)(z - m) and the given
// token's logit zt.  An empty row has lse = logp = -inf and entropy 0, a bad one NaN.
__device__ __forceinline__ void lp_finish(const LpOut &o, long long n, float m, double S, double T,
                                          float lnS, long long tok, long long V, float zt) {
  const float nan = __uint_as_float(0x7FC00000u);
  const bool bad = lnS != lnS, empty = lnS == -INFINITY;
  float lp, H, lse, mm = m;
  if (bad) {
    lp = H = lse = mm = nan;
  } else if (empty) {
    lp = lse = mm = -INFINITY;
    H = 0.f;
  } else {
    lp = (zt - m) - lnS;
    H = fmaxf(lnS - (float)(T / S), 0.f);
    lse = m + lnS;
  }
  if (tok < 0) lp = bad ? nan : 0.f;
  if (tok >= V) lp = nan;
  o.logp[n] = lp;
  o.entropy[n] = H;
  o.lse[n] = lse;
  if (o.stats) o.stats[n] = make_float2(mm, empty ? 0.f : lnS);
  if (o.status && (bad || tok >= V)) *o.status = o.bad_code;
}

// --- log probabilities from logits (kd_logprobs.hip) ---
constexpr int kLpMaxTop = 64;  // one alternative per lane of a wave
// Vocabulary splits of a row (1: no workspace and one launch).
int lp_splits(int64_t N, int64_t V, int dtype);
size_t lp_workspace(int64_t N, int64_t V, int32_t top, int dtype);
hipError_t launch_token_logprobs(int dtype, const void *logits, int64_t ld, const Tokens &tokens,
                                 int64_t N, int64_t V, int32_t top, const LpOut &out, void *ws,
                                 hipStream_t s);
// Upstream gradients may be null (zero).  dlogits may be logits itself when ld_d == ld.
struct LpGrad {
  const float2 *stats;
  const float *entropy, *g_logp, *g_entropy, *g_lse;
};
hipError_t launch_token_logprobs_bwd(int dtype, const void *logits, int64_t ld,
                                     const Tokens &tokens, int64_t N, int64_t V, const LpGrad &g,
                                     void *dlogits, int64_t ld_d, hipStream_t s);

// --- log probabilities from hidden states (kd_head.hip), one token chunk per call ---
// Partials per (head_part_rows vocabulary rows, token): part = (max, S), part_t = T in base 2.
int head_part_rows(int dtype, int64_t C, int64_t V);  // for chunks of C tokens
hipError_t launch_head_fwd(int dtype, const void *W, const void *h_c, int64_t rows, int64_t d,
                           int64_t V, const Tokens &tokens, float2 *part, float *part_t,
                           int64_t ld_part, int64_t C, float *zt, hipStream_t s);
// The same for at most kHeadFewTokens tokens (kd_head_few.hip): head_few_partials partials of
// each, one after the other (token r's from r * that on).
constexpr int64_t kHeadFewTokens = 64;
int64_t head_few_partials(int64_t N, int64_t V);
hipError_t launch_head_few(int dtype, const void *W, const void *h, int64_t rows, int64_t d,
                           int64_t V, const Tokens &tokens, float2 *part, float *part_t,
                           float *zt, hipStream_t s);
// Joins the partials (partial i of token r at i * ld + r, or for few at r * n_lse + i).
hipError_t launch_head_join(bool few, const float2 *part, const float *part_t, int64_t n_lse,
                            int64_t ld_part, int64_t rows, int64_t V, const float *zt,
                            const Tokens &tokens, const LpOut &out, hipStream_t s);
// Per token, what the gradient's epilogue reads: l2 = lse log2 e, and dz = p (a + b log2 p) +
// g [v = tok], tok -1 where there is none in range.
struct HeadTok {
  float l2, a, b, g;
  int tok;
};
__device__ __forceinline__ HeadTok head_tok(const Tokens &tokens, const LpGrad &g, int r, int V) {
  const long long tok = tokens.at(r);
  float gl = g.g_logp && tok >= 0 ? g.g_logp[r] : 0.f;
  if (tok >= V) gl = __uint_as_float(0x7FC00000u);
  const float ge = g.g_entropy ? g.g_entropy[r] : 0.f, gz = g.g_lse ? g.g_lse[r] : 0.f;
  const float2 st = g.stats[r];
  return {(float)(((double)st.x + (double)st.y) * 1.4426950408889634),
          (gz - gl) - ge * g.entropy[r], (float)(-(double)ge * kOpLn2d), gl,
          tok >= 0 && tok < V ? (int)tok : -1};
}
struct HeadCoef {  // per token of a chunk
  float *l2, *a, *b, *g;
  int *tok;
};
hipError_t launch_head_coef(const Tokens &tokens, const LpGrad &g, int64_t rows, int64_t V,
                            const HeadCoef &k, hipStream_t s);
// Few tokens in bf16: dz (null: not wanted; 2 * head_few_tokens * V_pad elements) in the order
// that launch_head_few_dh reads, and dW of type out (null: not wanted); V_pad a multiple of 256,
// ht as launch_transpose_h leaves it.  part: nsplit * head_few_tokens * (d rounded to 128).
inline int head_few_tokens(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
int head_few_dh_splits(int64_t d, int64_t V);
hipError_t launch_head_few_bwd(const void *W, const void *h, const void *ht, int64_t rows,
                               int64_t d, int64_t V, int64_t V_pad, const Tokens &tokens,
                               const LpGrad &g, void *dz, void *dW, int out, hipStream_t s);
hipError_t launch_head_few_dh(const void *W, const void *dz, int64_t rows, int64_t d, int64_t V,
                              int64_t V_pad, int nsplit, float *part, void *dh, hipStream_t s);
// dz as blocks of 256 vocabulary columns (element (c, v) at (v / 256) * C_alloc * 256 + c * 256
// + v % 256) and, bf16 and wanted, dzT (element (v, c) at (c / 256) * tst + v * 256 + c % 256).
hipError_t launch_head_dz(int dtype, const void *W, const void *h_c, int64_t rows, int64_t d,
                          int64_t V, const HeadCoef &k, void *dz, void *dzt, int64_t tst,
                          int64_t V_pad, int64_t C_alloc, hipStream_t s);

// Whether the dh product of a call with N tokens in chunks of C_alloc reads a k-contiguous copy
// of W (bf16), and into how many vocabulary splits (of k_split entries, a multiple of 256) it
// goes.
bool head_wt(int64_t N, int64_t C_alloc, int64_t d, int64_t V_pad);
void head_dh_splits(int dtype, bool wt, int64_t C_alloc, int64_t d, int64_t V_pad, int *nsplit,
                    int64_t *k_split);
// dh partials [nsplit][C_alloc][d_pad]; bf16 reads W through WT (launch_transpose_w), or itself
// where WT is null.
hipError_t launch_head_dh(int dtype, const void *dz, const void *W, const void *WT, int64_t rows,
                          int64_t d, int64_t V, int64_t V_pad, int nsplit, int64_t k_split,
                          float *part, int64_t d_pad, int64_t C_alloc, hipStream_t s);
// dW of type out = dz^T h over k tokens, plus old (float32, may be dW itself) where given.
hipError_t launch_head_dw(int dtype, int out, const void *dz, const void *dzt, const void *h_c,
                          const void *ht, int64_t k, int64_t d, int64_t V, int64_t V_pad,
                          int64_t C_alloc, const float *old, void *dW, hipStream_t s);

// --- gradient norm and clipping (kd_clip.hip) ---
// Float64 partials of the squares' sum (one per chunk of a tensor).
int64_t clip_partials(const int64_t *numel, int32_t n);
// scale false: the norm only.  outs null: in place.  Host arrays, read before the return.
hipError_t launch_clip_grads(const void *const *grads, void *const *outs, const int64_t *numel,
                             const int32_t *dtypes, int32_t n, bool scale, float max_norm,
                             float *norm, double *part, hipStream_t s);

}  // namespace kd
