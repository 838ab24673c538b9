// Log probabilities of given tokens from rows of logits, with the entropy, the logsumexp
// and the largest alternatives, and their gradient.
//
// For a row z with m = max z, S = sum exp(z - m), T = sum exp(z - m) (z - m):
//   lse = m + ln S,  ln p_v = z_v - m - ln S,  H = -sum p ln p = ln S - T / S.
// One pass: every lane keeps its own (m, S, T) and rescales the sums when its maximum
// rises; lanes, waves and vocabulary splits are joined by the same rule in double.
#include "kd_ops.h"

#include <cstdint>
#include <cstring>

namespace kd {
namespace {

constexpr int kLpThreads = 256, kLpWaves = kLpThreads / 64;
constexpr int kLpSlots = 4;  // 16-byte loads in flight per thread and step

template <int DT> struct LpT;
template <> struct LpT<1> { static constexpr int EPL = 8, ES = 2; };
template <> struct LpT<0> { static constexpr int EPL = 4, ES = 4; };

typedef unsigned int u4 __attribute__((ext_vector_type(4)));

// 16 bytes at any alignment of the element type (rows of an odd length or stride).
__device__ __forceinline__ u4 load16(const char *p) {
  u4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store16(char *p, u4 v) { __builtin_memcpy(p, &v, 16); }

template <int DT>
__device__ __forceinline__ void unpack(const u4 &r, float (&x)[LpT<DT>::EPL]) {
#pragma unroll
  for (int j = 0; j < LpT<DT>::EPL; ++j)
    x[j] = __uint_as_float(DT == 0 ? r[j]
                                   : (j & 1) ? (r[j >> 1] & 0xFFFF0000u) : (r[j >> 1] << 16));
}

// One group of EPL elements starting at element e: whole groups as 16 bytes, the last
// elements of a range one by one, -inf past the end (adds nothing, is no maximum).
template <int DT>
__device__ __forceinline__ u4 load_group(const char *row, long long e, long long end) {
  constexpr int EPL = LpT<DT>::EPL, ES = LpT<DT>::ES;
  if (e + EPL <= end) return load16(row + e * ES);
  const unsigned ninf = DT == 0 ? 0xFF800000u : 0xFF80FF80u;
  u4 r = {ninf, ninf, ninf, ninf};
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (e + j < end) {
      if (DT == 0) {
        r[j] = *(const unsigned *)(row + (e + j) * 4);
      } else {
        const unsigned h = *(const unsigned short *)(row + (e + j) * 2);
        r[j >> 1] = (j & 1) ? (r[j >> 1] & 0xFFFFu) | (h << 16) : (r[j >> 1] & 0xFFFF0000u) | h;
      }
    }
  return r;
}

// --- selection of the largest values -------------------------------------------------
// Order-preserving key of a float (-0 is +0), and back.
__device__ __forceinline__ unsigned val_key(float x) {
  unsigned u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_val(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// Value key, then the complemented index: unique, larger is better, equal values by
// rising index, so the result does not depend on timing.  0 is "none".
__device__ __forceinline__ uint64_t sel_key(float x, unsigned idx) {
  return ((uint64_t)val_key(x) << 32) | (unsigned)~idx;
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) {
  const unsigned lo = __shfl_xor((unsigned)v, o, 64), hi = __shfl_xor((unsigned)(v >> 32), o, 64);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint64_t shfl64(uint64_t v, int l) {
  const unsigned lo = __shfl((unsigned)v, l, 64), hi = __shfl((unsigned)(v >> 32), l, 64);
  return ((uint64_t)hi << 32) | lo;
}
// Bitonic sort of the wave's 64 keys, descending over the lanes.
template <class K, class X>
__device__ __forceinline__ K wave_sort(K v, int lane, X xchg) {
#pragma unroll
  for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const K o = xchg(v, j);
      const bool keep_max = ((lane & k) == 0) == ((lane & j) == 0);
      v = keep_max ? (v > o ? v : o) : (v < o ? v : o);
    }
  return v;
}
// The 64 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t wave_merge(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = shfl64(b, 63 - lane);
  uint64_t v = a > r ? a : r;  // bitonic
#pragma unroll
  for (int j = 32; j > 0; j >>= 1) {
    const uint64_t o = shfl_xor64(v, j);
    v = (lane & j) == 0 ? (v > o ? v : o) : (v < o ? v : o);
  }
  return v;
}

// A wave's running list of its 64 largest keys (one per lane, descending) with a buffer of
// candidates in LDS.  An element is a candidate if it reaches the threshold: the `top`-th
// largest so far (strictly above it once its slot is done: later elements of the wave have
// larger indices), or another wave's `top`-th value.
constexpr int kLpBuf = 128;
struct WaveTop {
  uint64_t list;
  float thr;
  int cnt, top, lane;
  volatile uint64_t *buf;
  __device__ __forceinline__ void init(int top_, int lane_, volatile uint64_t *b) {
    list = 0;
    thr = -INFINITY;
    cnt = 0;
    top = top_;
    lane = lane_;
    buf = b;
  }
  __device__ __forceinline__ void flush() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    while (cnt > 0) {
      const int n = cnt < 64 ? cnt : 64;
      uint64_t v = lane < n ? buf[cnt - n + lane] : 0ull;
      v = wave_sort(v, lane, [](uint64_t x, int o) { return shfl_xor64(x, o); });
      list = wave_merge(list, v, lane);
      cnt -= n;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  // The top-th value so far, -inf if there are fewer; strict: the next float above it.
  __device__ __forceinline__ void raise(bool strict) {
    const unsigned k = __builtin_amdgcn_readfirstlane(__shfl((unsigned)(list >> 32), top - 1, 64));
    if (k != 0) thr = fmaxf(thr, key_val(strict ? k + 1 : k));
  }
  __device__ __forceinline__ void offer(float x, unsigned idx, bool valid) {
    uint64_t mask = __builtin_amdgcn_ballot_w64(valid && x >= thr);
    if (mask == 0) return;
    if (cnt + __popcll(mask) > kLpBuf) {  // then the list is emptied, and at most 64 come in
      flush();
      raise(false);
      mask = __builtin_amdgcn_ballot_w64(valid && x >= thr);
    }
    if ((mask >> lane) & 1) {
      const int at = cnt + __builtin_amdgcn_mbcnt_hi((unsigned)(mask >> 32),
                                                     __builtin_amdgcn_mbcnt_lo((unsigned)mask, 0));
      buf[at] = sel_key(x, idx);
    }
    cnt += __popcll(mask);
  }
};

// Partial sums of one vocabulary split of a row.
struct LpPart {
  double S, T;
  float m;
  int pad;
};

// Joins (m2, S2, T2) to (m, S, T).  No value yet: m = -FLT_MAX, S = T = 0.
__device__ __forceinline__ void lp_join(float &m, double &S, double &T, float m2, double S2,
                                        double T2) {
  const float M = fmaxf(m, m2);
  const float d1 = fmaxf(m - M, kOpLowest), d2 = fmaxf(m2 - M, kOpLowest);
  const double c1 = (double)__builtin_amdgcn_exp2f(d1 * kOpLog2e);
  const double c2 = (double)__builtin_amdgcn_exp2f(d2 * kOpLog2e);
  T = c1 * (T + (double)d1 * S) + c2 * (T2 + (double)d2 * S2);
  S = c1 * S + c2 * S2;
  m = M;
}

struct LpArgs {
  const void *logits;
  long long ld, N, V;
  Tokens tokens;
  int top, S;
  long long per;  // elements of a split, a multiple of 8
  LpPart *part;   // [N][S] when S > 1
  uint64_t *keys; // [N][S][top]
  LpOut out;
};

// The row's alternatives from the sorted list (lane k holds the k-th).
__device__ __forceinline__ void write_top(const LpOut &o, long long row, int top, int lane,
                                          uint64_t key, float m, double lnS) {
  if (lane >= top) return;
  const float nan = __uint_as_float(0x7FC00000u);
  const bool bad = lnS != lnS, empty = lnS == -(double)INFINITY;
  const float x = key_val((unsigned)(key >> 32));
  o.top_idx[row * top + lane] = bad ? -1 : (int32_t)~(unsigned)key;
  o.top_logp[row * top + lane] =
      bad ? nan : empty ? -INFINITY : (float)((double)x - (double)m - lnS);
}

// One workgroup per (row, vocabulary split).
template <int DT, bool TOP>
__global__ __launch_bounds__(kLpThreads) void k_token_logprobs(LpArgs a) {
  constexpr int EPL = LpT<DT>::EPL, U = kLpSlots;
  __shared__ float s_m[kLpWaves];
  __shared__ double s_S[kLpWaves], s_T[kLpWaves];
  __shared__ volatile float s_thr[kLpWaves];
  __shared__ uint64_t s_buf[TOP ? kLpWaves * kLpBuf : 1];

  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const long long row = blockIdx.x / a.S;
  const int split = (int)(blockIdx.x - row * a.S);
  const long long e0 = split * a.per, end = e0 + a.per < a.V ? e0 + a.per : a.V;
  const char *rp = (const char *)a.logits + row * a.ld * LpT<DT>::ES;
  long long tok = -1;
  float zt = 0.f;
  if (t == 0 && a.S == 1) {
    tok = a.tokens.at(row);
    if (tok >= 0 && tok < a.V)
      zt = DT == 0 ? ((const float *)rp)[tok]
                   : __uint_as_float((unsigned)((const unsigned short *)rp)[tok] << 16);
  }

  float m = -3.4028234663852886e38f;
  double S = 0.0, T = 0.0;
  WaveTop wt;
  if (TOP) {
    wt.init(a.top, lane, s_buf + w * kLpBuf);
    if (lane == 0) s_thr[w] = -INFINITY;
    __syncthreads();
  }
  bool first = true;
  auto take = [&](const u4 (&raw)[U], long long base) {
    float x[U][EPL];
    float lu[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      unpack<DT>(raw[u], x[u]);
      lu[u] = x[u][0];
#pragma unroll
      for (int j = 1; j < EPL; ++j) lu[u] = fmaxf(lu[u], x[u][j]);
    }
    const float lm = fmaxf(fmaxf(lu[0], lu[1]), fmaxf(lu[2], lu[3]));
    if (lm > m) {
      const float d = fmaxf(m - lm, kOpLowest);
      const double c = (double)__builtin_amdgcn_exp2f(d * kOpLog2e);
      T = c * (T + (double)d * S);
      S = c * S;
      m = lm;
    }
    float ps = 0.f, pt = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const float d = x[u][j] - m;
        const float e = __builtin_amdgcn_exp2f(d * kOpLog2e);
        ps += e;
        pt = fmaf(e, fmaxf(d, kOpLowest), pt);
      }
    S += (double)ps;
    T += (double)pt;
    if (TOP) {
      if (first) {
        // the top-th largest of the 64 lanes' maxima: at least `top` elements reach it
        const unsigned k = wave_sort(val_key(lm), lane, [](unsigned v, int o) {
          return (unsigned)__shfl_xor(v, o, 64);
        });
        wt.thr = key_val(__builtin_amdgcn_readfirstlane(__shfl(k, a.top - 1, 64)));
        first = false;
      }
#pragma unroll
      for (int i = 0; i < kLpWaves; ++i) wt.thr = fmaxf(wt.thr, s_thr[i]);
      if (__builtin_amdgcn_ballot_w64(lm >= wt.thr)) {
        for (int u = 0; u < U; ++u) {
          if (!__builtin_amdgcn_ballot_w64(lu[u] >= wt.thr)) continue;
          const long long e = base + ((long long)u * kLpThreads + t) * EPL;
#pragma unroll
          for (int j = 0; j < EPL; ++j) wt.offer(x[u][j], (unsigned)(e + j), e + j < end);
        }
        if (wt.cnt >= 64) {
          wt.flush();
          wt.raise(false);
          if (lane == 0) s_thr[w] = wt.thr;
          wt.raise(true);
        }
      }
    }
  };

  // Whole steps are loaded one step ahead; the rest of the range is loaded with tests.
  constexpr long long STEP = (long long)kLpThreads * U * EPL;
  const long long whole = (end - e0) / STEP;
  u4 cur[U], nxt[U];
  const char *tp = rp + (e0 + (long long)t * EPL) * LpT<DT>::ES;
  if (whole > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) cur[u] = load16(tp + (size_t)u * kLpThreads * 16);
    for (long long i = 0; i < whole; ++i) {
      const long long n = i + 1 < whole ? i + 1 : i;  // the last step is loaded twice
#pragma unroll
      for (int u = 0; u < U; ++u)
        nxt[u] = load16(tp + (n * U + u) * (long long)(kLpThreads * 16));
      take(cur, e0 + i * STEP);
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = nxt[u];
    }
  }
  const long long rest = e0 + whole * STEP;
  if (rest < end) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      cur[u] = load_group<DT>(rp, rest + ((long long)u * kLpThreads + t) * EPL, end);
    take(cur, rest);
  }

  // lanes, then waves
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float m2 = __shfl_xor(m, o, 64);
    const double S2 = __shfl_xor(S, o, 64), T2 = __shfl_xor(T, o, 64);
    lp_join(m, S, T, m2, S2, T2);
  }
  if (lane == 0) {
    s_m[w] = m;
    s_S[w] = S;
    s_T[w] = T;
  }
  if (TOP) {
    wt.flush();
    s_buf[w * kLpBuf + lane] = wt.list;
  }
  __syncthreads();
  if (w != 0) return;
  for (int i = 1; i < kLpWaves; ++i) {
    lp_join(m, S, T, s_m[i], s_S[i], s_T[i]);
    if (TOP) wt.list = wave_merge(wt.list, s_buf[i * kLpBuf + lane], lane);
  }
  if (a.S > 1) {
    const long long at = row * a.S + split;
    if (lane == 0) a.part[at] = LpPart{S, T, m, 0};
    if (TOP && lane < a.top) a.keys[at * a.top + lane] = wt.list;
    return;
  }
  double lnS = 0.0;
  if (lane == 0) lnS = lp_finish(a.out, row, m, S, T, tok, a.V, zt);
  if (TOP) write_top(a.out, row, a.top, lane, wt.list, m, __shfl(lnS, 0, 64));
}

// Joins a row's vocabulary splits: one workgroup per row.
template <int DT, bool TOP>
__global__ __launch_bounds__(kLpThreads) void k_token_logprobs_join(LpArgs a) {
  __shared__ uint64_t s_list[TOP ? kLpThreads : 1];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const long long row = blockIdx.x;
  uint64_t list = 0;
  if (TOP) {
    for (int i = w; i < a.S; i += kLpWaves) {
      const uint64_t v = lane < a.top ? a.keys[(row * a.S + i) * a.top + lane] : 0ull;
      list = wave_merge(list, v, lane);
    }
    s_list[t] = list;
    __syncthreads();
  }
  if (w != 0) return;
  if (TOP)
    for (int i = 1; i < kLpWaves; ++i) list = wave_merge(list, s_list[i * 64 + lane], lane);
  float m = -3.4028234663852886e38f;
  double S = 0.0, T = 0.0;
  for (int i = lane; i < a.S; i += 64) {
    const LpPart p = a.part[row * a.S + i];
    lp_join(m, S, T, p.m, p.S, p.T);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float m2 = __shfl_xor(m, o, 64);
    const double S2 = __shfl_xor(S, o, 64), T2 = __shfl_xor(T, o, 64);
    lp_join(m, S, T, m2, S2, T2);
  }
  double lnS = 0.0;
  if (lane == 0) {
    const long long tok = a.tokens.at(row);
    float zt = 0.f;
    const char *rp = (const char *)a.logits + row * a.ld * LpT<DT>::ES;
    if (tok >= 0 && tok < a.V)
      zt = DT == 0 ? ((const float *)rp)[tok]
                   : __uint_as_float((unsigned)((const unsigned short *)rp)[tok] << 16);
    lnS = lp_finish(a.out, row, m, S, T, tok, a.V, zt);
  }
  if (TOP) write_top(a.out, row, a.top, lane, list, m, __shfl(lnS, 0, 64));
}

// dz_v = p_v (g_lse - g_logp - g_entropy (ln p_v + H)) + g_logp [v = t], one thread per
// 16-byte group: one read and one write of the row, nothing between.
struct LpBwdArgs {
  const void *logits;
  long long ld, N, V;
  Tokens tokens;
  LpGrad g;
  void *out;
  long long ld_d;
  unsigned segs;  // workgroups per row
};

template <int DT>
__global__ __launch_bounds__(kLpThreads) void k_token_logprobs_bwd(LpBwdArgs a) {
  constexpr int EPL = LpT<DT>::EPL, ES = LpT<DT>::ES, U = kLpSlots;
  const long long row = blockIdx.x / a.segs;
  const unsigned seg = blockIdx.x - (unsigned)row * a.segs;
  const char *rp = (const char *)a.logits + row * a.ld * ES;
  char *wp = (char *)a.out + row * a.ld_d * ES;
  const long long e0 = ((long long)seg * U * kLpThreads + threadIdx.x) * EPL;
  u4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    raw[u] = load_group<DT>(rp, e0 + (long long)u * kLpThreads * EPL, a.V);
  const float2 st = a.g.stats[row];
  const long long tok = a.tokens.at(row);
  float gl = a.g.g_logp && tok >= 0 ? a.g.g_logp[row] : 0.f;
  if (tok >= a.V) gl = __uint_as_float(0x7FC00000u);
  const float ge = a.g.g_entropy ? a.g.g_entropy[row] : 0.f;
  const float gz = a.g.g_lse ? a.g.g_lse[row] : 0.f;
  const float c = (gz - gl) - ge * a.g.entropy[row];
  const bool empty = st.x == -INFINITY;
  const long long hot = gl == 0.f || empty ? -1 : tok;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long e = e0 + (long long)u * kLpThreads * EPL;
    if (e >= a.V) break;
    float x[EPL];
    unpack<DT>(raw[u], x);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float lp = (x[j] - st.x) - st.y;  // ln p
      const float p = __builtin_amdgcn_exp2f(lp * kOpLog2e);
      x[j] = empty ? 0.f : p * fmaf(-ge, fmaxf(lp, kOpLowest), c);
      if (e + j == hot) x[j] += gl;
    }
    u4 r;
    if (DT == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = __float_as_uint(x[j]);
    } else {
      typedef __bf16 b2 __attribute__((ext_vector_type(2)));
      typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int j = 0; j < 4; ++j)  // one rounding, to nearest even
        r[j] = __builtin_bit_cast(unsigned, __builtin_convertvector(
                                                f2{x[(2 * j) % EPL], x[(2 * j + 1) % EPL]}, b2));
    }
    if (e + EPL <= a.V) {
      store16(wp + e * ES, r);
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (e + j < a.V) {
          if (DT == 0) *(unsigned *)(wp + (e + j) * 4) = r[j % 4];
          else *(unsigned short *)(wp + (e + j) * 2) =
              (unsigned short)((j & 1) ? r[j >> 1] >> 16 : r[j >> 1] & 0xFFFFu);
        }
    }
  }
}

inline int64_t cd(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

int lp_splits(int64_t N, int64_t V, int) {
  const int64_t want = N > 0 ? 1024 / N : 1, most = cd(V, 4096);
  int64_t s = want < most ? want : most;
  if (s > 64) s = 64;
  return s < 1 ? 1 : (int)s;
}

size_t lp_workspace(int64_t N, int64_t V, int32_t top, int dtype) {
  const int64_t S = lp_splits(N, V, dtype);
  return S == 1 ? 0 : (size_t)(N * S) * (sizeof(LpPart) + 8 * (size_t)top);
}

hipError_t launch_token_logprobs(int dtype, const void *logits, int64_t ld, const Tokens &tokens,
                                 int64_t N, int64_t V, int32_t top, const LpOut &out, void *ws,
                                 hipStream_t s) {
  if (N <= 0) return hipSuccess;
  const int S = lp_splits(N, V, dtype);
  LpArgs a{logits, ld, N, V, tokens, top, S, cd(cd(V, S), 8) * 8, nullptr, nullptr, out};
  if (S > 1) {
    a.part = (LpPart *)ws;
    a.keys = (uint64_t *)((char *)ws + (size_t)N * S * sizeof(LpPart));
  }
  const dim3 grid((unsigned)(N * S)), block(kLpThreads), rows((unsigned)N);
#define KD_LP(DT, TOP)                                                                  \
  do {                                                                                  \
    hipLaunchKernelGGL((k_token_logprobs<DT, TOP>), grid, block, 0, s, a);              \
    if (S > 1)                                                                          \
      hipLaunchKernelGGL((k_token_logprobs_join<DT, TOP>), rows, block, 0, s, a);       \
  } while (0)
  if (dtype == 1) {
    if (top > 0) KD_LP(1, true);
    else KD_LP(1, false);
  } else {
    if (top > 0) KD_LP(0, true);
    else KD_LP(0, false);
  }
#undef KD_LP
  return hipGetLastError();
}

hipError_t launch_token_logprobs_bwd(int dtype, const void *logits, int64_t ld,
                                     const Tokens &tokens, int64_t N, int64_t V, const LpGrad &g,
                                     void *dlogits, int64_t ld_d, hipStream_t s) {
  if (N <= 0) return hipSuccess;
  const int64_t epl = dtype == 1 ? 8 : 4;
  LpBwdArgs a{logits, ld, N, V, tokens, g, dlogits, ld_d,
              (unsigned)cd(V, epl * kLpSlots * kLpThreads)};
  const dim3 grid((unsigned)(N * a.segs)), block(kLpThreads);
  if (dtype == 1)
    hipLaunchKernelGGL(k_token_logprobs_bwd<1>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(k_token_logprobs_bwd<0>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace kd
