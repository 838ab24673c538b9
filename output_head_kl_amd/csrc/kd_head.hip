// Log probabilities of given tokens from hidden states, z = h W^T with no logits in memory,
// and their gradients.  The products run on the MFMA GEMM core (kd_gemm.h) over one token
// chunk at a time; these are its epilogues and the row kernels around it.
//
//  forward   per (token, wave row of the vocabulary tile): max, S = sum 2^t, T2 = sum t 2^t
//            with t = (z - max) log2 e, and the given token's z straight from the lane that
//            holds it; k_head_join folds the partials into logp, entropy and lse.
//  gradient  z again, then dz = p (gz - gl - ge (ln p + H)) + gl [v = t] in one rounding, in
//            the layouts the dh and dW GEMMs of the loss read.
//
// Up to 64 tokens go the ways of kd_head_few.hip.  Above, the products bound the time: 4096
// tokens, d 2880, V 201088 in bf16 take 3.5 ms forward (1350 TFLOP/s) and 12.0 ms for the
// gradients: z again 3.9, dh 3.6 with the partials' sum, W's copy for it 0.5, dW 4.0.
#include "kd_gemm.h"
#include "kd_gemm32.h"
#include "kd_ops.h"

namespace kd {
namespace {

// Tile rows are vocabulary entries v, columns tokens c (layouts as in kd_gemm.h).
template <int DT>
struct EpiHeadFwd {
  static constexpr bool kPrefetch = false;
  struct Pre {};
  float2 *part;     // [n_lse][ld] (max, S)
  float *part_t;    // [n_lse][ld] T2
  long long ld;
  int V, rows;
  Tokens tokens;    // of the chunk
  float *zt;        // [rows] the given tokens' logits
  template <int NRB, int NCB>
  __device__ __forceinline__ void operator()(f32x16 (&acc)[NRB][NCB], int m0, int n0, int lane,
                                             int, char *) const {
    constexpr int WR = 32 * NRB;
    if (m0 >= V) return;
    const int vl = m0 + (lane >> 5) * 4;
    const bool full = m0 + WR <= V;
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) {
      const int c = n0 + cb * 32 + (lane & 31);
      const long long rel = c < rows ? tokens.at(c) - m0 : -1;  // the token's row in the wave
      const int r = rel >= 0 && rel < WR && rel < V - m0 ? (int)rel : -1;
      if (__builtin_amdgcn_ballot_w64(r >= 0)) {
        // few waves hold a given token: the lane and accumulator with its row
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (rb * 32 + (i >> 2) * 8 + (lane >> 5) * 4 + (i & 3) == r) zt[c] = acc[rb][cb][i];
      }
      float mx = -INFINITY;
      if (full) {
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
          for (int i = 0; i < 16; ++i) mx = fmaxf(mx, acc[rb][cb][i]);
      } else {
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (vl + rb * 32 + (i >> 2) * 8 + (i & 3) < V) mx = fmaxf(mx, acc[rb][cb][i]);
      }
      mx = halves_max(mx);
      if (!full) {
        // rows past the vocabulary: so far below the maximum that 2^t is 0, and finite
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (vl + rb * 32 + (i >> 2) * 8 + (i & 3) >= V) acc[rb][cb][i] = mx + kOpLowest;
      }
      const float mx2 = mx * kLog2e;
      float s = 0.f, t2 = 0.f;
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float t = fmaf(acc[rb][cb][i], kLog2e, -mx2);
          const float e = fast_exp2(t);
          s += e;
          t2 = fmaf(e, t, t2);
        }
      s = halves_sum(s);
      t2 = halves_sum(t2);
      if (lane < 32 && c < rows) {
        part[(long long)(m0 / WR) * ld + c] = make_float2(mx, s);
        part_t[(long long)(m0 / WR) * ld + c] = t2;
      }
    }
  }
};

// Joins a token's partials, in a fixed order: TOK tokens per workgroup (8, for 64-byte reads
// where a partial's tokens lie side by side; 1 where a token's partials do), 1024 / TOK
// threads per token, each up to eight partials at a time; then lanes, then waves.  Reads 12
// bytes per partial: 24 us for 4096 tokens of 1048 partials (2.1 TB/s), 5 us, a launch's
// latency, for 48.
constexpr int kJoinThreads = 1024;
__device__ __forceinline__ void head_join(float &m, double &S, double &T, float m2, double S2,
                                          double T2) {
  const float M = __builtin_elementwise_maximum(m, m2);  // NaN stays
  const float d1 = fmaxf(m - M, kOpLowest), d2 = fmaxf(m2 - M, kOpLowest);
  const double c1 = (double)fast_exp2(d1 * kLog2e), c2 = (double)fast_exp2(d2 * kLog2e);
  T = c1 * (T + (double)d1 * S) + c2 * (T2 + (double)d2 * S2);
  S = c1 * S + c2 * S2;
  m = M;
}
template <int TOK>
__global__ __launch_bounds__(kJoinThreads) void k_head_join(const float2 *part,
                                                            const float *part_t, int n_lse,
                                                            long long si, long long sr, int rows,
                                                            int V, const float *zt, Tokens tokens,
                                                            LpOut out) {
  constexpr int NW = kJoinThreads / 64, SLOTS = kJoinThreads / TOK, U = 8;
  constexpr float kNone = -3.4028234663852886e38f;
  __shared__ float sm[NW * TOK];
  __shared__ double sS[NW * TOK], sT[NW * TOK];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, slot = t / TOK;
  const int r = blockIdx.x * TOK + t % TOK;
  float m = kNone;
  double S = 0.0, T = 0.0;
  if (r < rows)
    for (int i0 = slot; i0 < n_lse; i0 += U * SLOTS) {
      float2 q[U];
      float t2[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * SLOTS;
        q[u] = i < n_lse ? part[i * si + r * sr] : make_float2(kNone, 0.f);
        t2[u] = i < n_lse ? part_t[i * si + r * sr] : 0.f;
      }
      float M = q[0].x;
#pragma unroll
      for (int u = 1; u < U; ++u) M = __builtin_elementwise_maximum(M, q[u].x);
      float s = 0.f, tt = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float d = fmaxf(q[u].x - M, kOpLowest), c = fast_exp2(d * kLog2e);
        s = fmaf(c, q[u].y, s);
        tt = fmaf(c, fmaf(t2[u], (float)kOpLn2d, d * q[u].y), tt);
      }
      head_join(m, S, T, M, (double)s, (double)tt);
    }
  auto lanes = [&](int from) {
#pragma unroll
    for (int o = TOK; o < 64; o <<= 1) {
      if (o >= from) break;
      const float m2 = __shfl_xor(m, o, 64);
      const double S2 = __shfl_xor(S, o, 64), T2 = __shfl_xor(T, o, 64);
      head_join(m, S, T, m2, S2, T2);
    }
  };
  lanes(64);
  if (lane < TOK) {
    sm[w * TOK + lane] = m;
    sS[w * TOK + lane] = S;
    sT[w * TOK + lane] = T;
  }
  __syncthreads();
  if (w != 0) return;
  // NW * TOK entries: two per lane, or one for the first of them
  constexpr int E = NW * TOK;
  const int e = lane % E;
  m = sm[e];
  S = sS[e];
  T = sT[e];
  static_assert(E == 128 || E == 16, "entries of the first wave");
  if (E == 128) head_join(m, S, T, sm[e + E / 2], sS[e + E / 2], sT[e + E / 2]);
  lanes(E < 64 ? E : 64);
  if (lane >= TOK || r >= rows) return;
  const long long tok = tokens.at(r);
  if (T != T) S = T;  // a logit that is not finite
  lp_finish(out, r, m, S, T, lp_log(m, S), tok, V, tok >= 0 && tok < V ? zt[r] : 0.f);
}

__global__ void k_head_coef(Tokens tokens, LpGrad g, int rows, int V, HeadCoef k) {
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= rows) return;
  const HeadTok c = head_tok(tokens, g, r, V);
  k.l2[r] = c.l2;
  k.a[r] = c.a;
  k.b[r] = c.b;
  k.g[r] = c.g;
  k.tok[r] = c.tok;
}

template <int DT>
struct EpiHeadDz {
  static constexpr bool kPrefetch = false;
  struct Pre {};
  void *dz;      // blocks of 256 vocabulary columns: [V_pad/256][C_alloc][256]
  long long ts;  // C_alloc * 256
  const float *l2, *a, *b, *gt;
  const int *tok;
  int V, rows, V_pad;
  unsigned short *dzt;  // bf16, or null: (v, c) at dzt[(c / 256) * tst + v * 256 + c % 256]
  long long tst;
  template <int NRB, int NCB>
  __device__ __forceinline__ void operator()(f32x16 (&acc)[NRB][NCB], int m0, int n0, int lane,
                                             int, char *smem) const {
    const int vl = m0 + (lane >> 5) * 4;
    if (m0 + 32 * NRB > V) {
      // rows V <= v < V_pad get p = 0 and a finite factor: dz = 0
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (vl + rb * 32 + (i >> 2) * 8 + (i & 3) >= V) {
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb) acc[rb][cb][i] = -1e30f;
          }
    }
    if constexpr (DT == 1) staged(acc, m0, n0, lane, smem);
    else direct(acc, m0, n0, lane);
  }

  // One element: log2 p, p, then the formula; g is the given token's extra term or 0.
  static __device__ __forceinline__ float one(float z, float l2, float a, float b, float g) {
    const float q = fmaf(z, kLog2e, -l2);
    return fmaf(fast_exp2(q), fmaf(b, q, a), g);
  }

  // fp32: four rows of a token at a time.
  template <int NRB, int NCB>
  __device__ __forceinline__ void direct(const f32x16 (&acc)[NRB][NCB], int m0, int n0,
                                         int lane) const {
    const int vl = m0 + (lane >> 5) * 4;
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) {
      const int c = n0 + cb * 32 + (lane & 31);
      if (c >= rows) continue;
      const float cl2 = l2[c], ca = a[c], cbb = b[c], cg = gt[c];
      const int ct = tok[c];
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int v0 = vl + rb * 32 + g * 8;
          if (v0 >= V_pad) continue;  // V_pad is a multiple of 4
          f32x4 x;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = one(acc[rb][cb][g * 4 + e], cl2, ca, cbb, v0 + e == ct ? cg : 0.f);
          *(f32x4 *)((float *)dz + (long long)(v0 >> 8) * ts + c * 256 + (v0 & 255)) = x;
        }
    }
  }

  // bf16: through a per-wave LDS slice of [32 NCB tokens][64 rows] per pass, so that dz leaves
  // as whole 128-byte lines of a token's rows and dzT as 16-byte pieces (8 tokens) of a row.
  // The given token's element is written again in the slice, from its float32 value.
  template <int NRB, int NCB>
  __device__ __forceinline__ void staged(const f32x16 (&acc)[NRB][NCB], int m0, int n0, int lane,
                                         char *smem) const {
    constexpr int RP = 2, NP = NRB / RP;                 // 32-row blocks per pass, passes
    constexpr int TOK = 32 * NCB, PITCH = RP * 32 + 8;   // tokens per wave, bf16 per row
    constexpr int QPR = RP * 32 / 8;                     // 16-byte pieces per token row
    constexpr int TG = TOK / 8;                          // 8-token groups per vocabulary row
    static_assert(NRB % RP == 0, "whole passes");
    __syncthreads();  // every wave is done with the k-loop's LDS ring
    LDS_AS unsigned short *stg =
        (LDS_AS unsigned short *)smem + (threadIdx.x >> 6) * TOK * PITCH;
    float cl2[NCB], ca[NCB], cbb[NCB], cg[NCB];
    int ct[NCB];  // the given token's row in the wave, or out of range
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) {
      // tokens rows <= c < C_alloc get zeros: the dW GEMM reads dzT in 8-token chunks
      const int c = n0 + cb * 32 + (lane & 31);
      const bool cv = c < rows;
      cl2[cb] = cv ? l2[c] : 0.f;
      ca[cb] = cv ? a[c] : 0.f;
      cbb[cb] = cv ? b[c] : 0.f;
      cg[cb] = cv ? gt[c] : 0.f;
      const int t = cv ? tok[c] : -1;
      ct[cb] = t >= m0 && t - m0 < 32 * NRB ? t - m0 : -1;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb) {
        const int cl = cb * 32 + (lane & 31);
#pragma unroll
        for (int r = 0; r < RP; ++r)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = one(acc[p * RP + r][cb][g * 4 + e], cl2[cb], ca[cb], cbb[cb], 0.f);
            const u32x2 pk = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
            *(LDS_AS u32x2 *)(stg + cl * PITCH + r * 32 + g * 8 + (lane >> 5) * 4) = pk;
          }
        const int hr = ct[cb] - p * RP * 32;
        if (__builtin_amdgcn_ballot_w64(hr >= 0 && hr < RP * 32)) {
#pragma unroll
          for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int row = r * 32 + (i >> 2) * 8 + (lane >> 5) * 4 + (i & 3);
              if (row == hr)
                stg[cl * PITCH + row] = f32_to_bf16(
                    one(acc[p * RP + r][cb][i], cl2[cb], ca[cb], cbb[cb], cg[cb]));
            }
        }
      }
      const int vp = m0 + p * RP * 32;  // first vocabulary row of the pass
#pragma unroll
      for (int it = 0; it < TOK * QPR / 64; ++it) {
        const int q = it * 64 + lane, cl = q / QPR, pc = q - cl * QPR;
        const int c = n0 + cl, v = vp + pc * 8;
        const u32x4 val = *(const LDS_AS u32x4 *)(stg + cl * PITCH + pc * 8);
        if (c < rows && v < V_pad)
          *(u32x4 *)((unsigned short *)dz + (long long)(v >> 8) * ts + c * 256 + (v & 255)) = val;
      }
      if (!dzt) continue;
#pragma unroll
      for (int it = 0; it < RP * 32 * TG / 64; ++it) {
        const int q = it * 64 + lane, r = q / TG, tg = q - r * TG;
        const int v = vp + r;
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = (unsigned)stg[(tg * 8 + 2 * e) * PITCH + r] |
                 ((unsigned)stg[(tg * 8 + 2 * e + 1) * PITCH + r] << 16);
        const int c = n0 + tg * 8;
        if (v < V_pad)
          __builtin_nontemporal_store(
              o, (u32x4 *)(dzt + (long long)(c >> 8) * tst + (long long)v * 256 + (c & 255)));
      }
    }
  }
};

// dh partials of one vocabulary split: tile rows are hidden units j, columns tokens c.
struct EpiHeadDh {
  static constexpr bool kPrefetch = false;
  struct Pre {};
  float *part;
  long long split_stride, ld;  // C_alloc * d_pad, d_pad
  int rows;
  template <int NRB, int NCB>
  __device__ __forceinline__ void operator()(f32x16 (&acc)[NRB][NCB], int m0, int n0, int lane,
                                             int split, char *) const {
    const int jl = m0 + (lane >> 5) * 4;
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) {
      const int c = n0 + cb * 32 + (lane & 31);
      if (c >= rows) continue;
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int j = jl + rb * 32 + g * 8;
          if (j >= ld) continue;  // d_pad is a multiple of 4
          *(f32x4 *)(part + split * split_stride + c * ld + j) =
              f32x4{acc[rb][cb][g * 4], acc[rb][cb][g * 4 + 1], acc[rb][cb][g * 4 + 2],
                    acc[rb][cb][g * 4 + 3]};
        }
    }
  }
};

// dW: tile rows are vocabulary entries v, columns hidden units j; the sum over one group of
// tokens plus, where `old` is given, what earlier groups left there (each element belongs to
// one lane of one launch).  bf16 is rounded once, here: lanes l and l ^ 1 swap halves of two
// rows, so that each stores two neighbouring columns of one of them.
template <int OUT>
struct EpiHeadDw {
  static constexpr bool kPrefetch = false;
  struct Pre {};
  void *dW;
  const float *old;
  int d, V;
  template <int NRB, int NCB>
  __device__ __forceinline__ void operator()(f32x16 (&acc)[NRB][NCB], int m0, int n0, int lane,
                                             int, char *) const {
    const int vl = m0 + (lane >> 5) * 4;
    const bool odd = lane & 1;
#pragma unroll
    for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int v = vl + rb * 32 + (i >> 2) * 8 + (i & 3);
        if (v >= V) continue;
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb) {
          const int j = n0 + cb * 32 + (lane & 31);
          float x0 = acc[rb][cb][i], x1 = acc[rb][cb][i + 1];
          if (old && j < d) {
            x0 += old[(long long)v * d + j];
            if (v + 1 < V) x1 += old[(long long)(v + 1) * d + j];
          }
          if constexpr (OUT == 0) {
            if (j < d) {
              ((float *)dW)[(long long)v * d + j] = x0;
              if (v + 1 < V) ((float *)dW)[(long long)(v + 1) * d + j] = x1;
            }
          } else {
            // d is a multiple of 8: both columns of a pair are inside or neither
            const float got = __uint_as_float(__builtin_amdgcn_update_dpp(
                0u, __float_as_uint(odd ? x0 : x1), 0xB1, 0xF, 0xF, true));
            const unsigned pk = odd ? pack_bf16x2(got, x1) : pack_bf16x2(x0, got);
            const int r = v + (odd ? 1 : 0);
            if (j < d && r < V)
              *(unsigned *)((unsigned short *)dW + (long long)r * d + (j & ~1)) = pk;
          }
        }
      }
  }
};

// Rows of a bf16 tile of an m x n product of k-contiguous operands, one workgroup per compute
// unit at a time.  384 are 13 % faster per row (4096 tokens, d 4096, V 128256 forward: 3.14
// against 3.56 ms), but 256 leave less of the last round empty (256 tokens of them: 264 against
// 325 us; 1024 tokens, d 1024, V 32000: 72 against 88).
constexpr double kRowGain = 1.13;
int tile16(int64_t m, int64_t n) {
  auto rounds = [&](int64_t t) { return (((m + t - 1) / t) * ((n + kTile - 1) / kTile) + 255) / 256; };
  return kRowGain * (double)(rounds(256) * 256) < (double)(rounds(384) * 384) ? 256 : 384;
}
// The same for the dh product, whose splits fill the rounds: what counts is rows past d.
int dh_tile16(int64_t d) {
  const int64_t r2 = (d + 255) / 256 * 256, r3 = (d + 383) / 384 * 384;
  return kRowGain * (double)r2 < (double)r3 ? 256 : 384;
}

// G.ntm counts tiles of T rows.
template <class Epi>
hipError_t run16(int T, const Operand &A, const Operand &B, const GemmGrid &G, const Epi &epi,
                 hipStream_t s) {
  if (T == kTileA16) return run_gemm<1, OP_KC, OP_KC>(A, B, G, epi, s);
  hipLaunchKernelGGL((gemm_pipe_kernel<OP_KC, OP_KC, Epi, 2, 2, 64, 4, 256>),
                     dim3((unsigned)((long long)G.ntm * G.ntn * G.nsplit)), dim3(512), 0, s, A, B,
                     G, epi);
  return hipGetLastError();
}

}  // namespace

int head_part_rows(int dtype, int64_t C, int64_t V) {
  return (dtype == 1 ? tile16(V, C) : g32::tile(V, C, 1)) / 2;
}

hipError_t launch_head_fwd(int dtype, const void *W, const void *h_c, int64_t rows, int64_t d,
                           int64_t V, const Tokens &tokens, float2 *part, float *part_t,
                           int64_t ld_part, int64_t C, float *zt, hipStream_t s) {
  Operand A{W, d, (int)V, (int)d, 256};
  Operand B{h_c, d, (int)rows, (int)d, 256};
  if (dtype == 1) {
    // token tiles in groups of eight: an XCD's concurrent workgroups then share four
    // vocabulary tiles and eight token tiles
    const int T = tile16(V, C);  // of all chunks: the partials' places depend on it
    GemmGrid G{cdiv(V, T), cdiv(rows, kTile), 1, (int)d, (int)d, 0, 8};
    EpiHeadFwd<1> e{part, part_t, ld_part, (int)V, (int)rows, tokens, zt};
    return run16(T, A, B, G, e, s);
  }
  EpiHeadFwd<0> e{part, part_t, ld_part, (int)V, (int)rows, tokens, zt};
  return g32::run<OP_KC, OP_KC>(g32::tile(V, C, 1), V, rows, 1, d, d, A, B, e, s);
}

hipError_t launch_head_join(bool few, const float2 *part, const float *part_t, int64_t n_lse,
                            int64_t ld_part, int64_t rows, int64_t V, const float *zt,
                            const Tokens &tokens, const LpOut &out, hipStream_t s) {
  if (few)
    hipLaunchKernelGGL(k_head_join<1>, dim3((unsigned)rows), dim3(kJoinThreads), 0, s, part,
                       part_t, (int)n_lse, 1LL, (long long)n_lse, (int)rows, (int)V, zt, tokens,
                       out);
  else
    hipLaunchKernelGGL(k_head_join<8>, dim3(cdiv(rows, 8)), dim3(kJoinThreads), 0, s, part, part_t,
                       (int)n_lse, (long long)ld_part, 1LL, (int)rows, (int)V, zt, tokens, out);
  return hipGetLastError();
}

hipError_t launch_head_coef(const Tokens &tokens, const LpGrad &g, int64_t rows, int64_t V,
                            const HeadCoef &k, hipStream_t s) {
  hipLaunchKernelGGL(k_head_coef, dim3(cdiv(rows, 256)), dim3(256), 0, s, tokens, g, (int)rows,
                     (int)V, k);
  return hipGetLastError();
}

hipError_t launch_head_dz(int dtype, const void *W, const void *h_c, int64_t rows, int64_t d,
                          int64_t V, const HeadCoef &k, void *dz, void *dzt, int64_t tst,
                          int64_t V_pad, int64_t C_alloc, hipStream_t s) {
  // vocabulary tiles cover V_pad, so that dz holds zeros from V on
  Operand A{W, d, (int)V, (int)d, 256};
  Operand B{h_c, d, (int)rows, (int)d, 256};
  if (dtype == 1) {
    const int T = tile16(V_pad, rows);  // V_pad is a multiple of both
    GemmGrid G{(int)(V_pad / T), cdiv(rows, kTile), 1, (int)d, (int)d, 0, 8};
    EpiHeadDz<1> e{dz, C_alloc * 256, k.l2, k.a, k.b, k.g, k.tok, (int)V, (int)rows, (int)V_pad,
                   (unsigned short *)dzt, tst};
    return run16(T, A, B, G, e, s);
  }
  EpiHeadDz<0> e{dz, C_alloc * 256, k.l2, k.a, k.b, k.g, k.tok, (int)V, (int)rows, (int)V_pad,
                 nullptr, 0};
  return g32::run<OP_KC, OP_KC>(g32::tile(V_pad, rows, 1), V_pad, rows, 1, d, d, A, B, e, s);
}

// The float32 tile of the dh product, which has up to 32 splits to fill the chip.
static int dh_tile32(int64_t C_alloc, int64_t d) { return g32::tile(d, C_alloc, 32); }

// Enough splits of the vocabulary to fill whole rounds of the workgroups that run at once (one
// per compute unit in bf16, two in float32); more only where they fill the rounds 5 % better,
// as each adds a float32 partial of dh.
void head_dh_splits(int dtype, bool wt, int64_t C_alloc, int64_t d, int64_t V_pad, int *nsplit,
                    int64_t *k_split) {
  const int64_t C = C_alloc, t32 = dh_tile32(C_alloc, d);
  const int64_t tm = dtype == 1 ? (wt ? dh_tile16(d) : kTile) : t32, tn = dtype == 1 ? kTile : t32;
  const int64_t tiles = ((d + tm - 1) / tm) * ((C + tn - 1) / tn), slots = dtype == 1 ? 256 : 512;
  int64_t ns = 1;
  double best = 0.0;
  for (int64_t c = 1; c <= 32 && c <= V_pad / kTile; ++c) {
    const int64_t wgs = tiles * c, rounds = (wgs + slots - 1) / slots;
    const double fill = (double)wgs / (double)(rounds * slots);
    if ((rounds == 1 && fill > best) || fill > best + 0.05) {
      best = fill;
      ns = c;
    }
  }
  *k_split = ((V_pad + ns - 1) / ns + kTile - 1) / kTile * kTile;
  *nsplit = (int)((V_pad + *k_split - 1) / *k_split);
}

// The copy costs a read and a write of W, and lets the dh product read both operands without
// transposing them in LDS, on a 384-row tile.  Up to 1024 tokens it does not pay (512, d 4096, V
// 128256: all gradients 2.10 ms with it, 1.76 without), above 4096 it does (16384, 2048, 128256:
// 21.8 and 23.7 ms).  Between, the two are compared in units of the product without it on a full
// chip, 18 % longer there: what the rounds leave empty (which measured more than its share,
// hence the power), rows past d, and the copy, 580 / N.  2048 tokens, d 1024, V 32000: 529 and
// 431 us; 4096, 2880, 201088: 12.1 and 13.4 ms.
bool head_wt(int64_t N, int64_t C_alloc, int64_t d, int64_t V_pad) {
  if (N <= 1024 || N > 4096) return N > 4096;
  auto cost = [&](bool wt) {
    int ns;
    int64_t ks;
    head_dh_splits(1, wt, C_alloc, d, V_pad, &ns, &ks);
    const int64_t tm = wt ? dh_tile16(d) : kTile, rows = (d + tm - 1) / tm * tm;
    const int64_t tiles = rows / tm * (C_alloc / kTile), rounds = (tiles * ns + 255) / 256;
    const double e = (double)(V_pad * tiles) / (double)(rounds * 256 * ks);
    const double t = (double)rows / (double)d / (e * e * e * e);
    if (!wt) return rounds == 1 ? t : 1.12 * t;
    return t / (tm == kTile ? 1.18 / kRowGain : 1.18) + 580.0 / (double)N;
  };
  return cost(true) < cost(false);
}

// D[j][c] = sum_v W[v][j] dz[c][v]
hipError_t launch_head_dh(int dtype, const void *dz, const void *W, const void *WT, int64_t rows,
                          int64_t d, int64_t V, int64_t V_pad, int nsplit, int64_t k_split,
                          float *part, int64_t d_pad, int64_t C_alloc, hipStream_t s) {
  Operand B{dz, 256, (int)rows, (int)V_pad, C_alloc * 256};
  EpiHeadDh e{part, C_alloc * d_pad, d_pad, (int)rows};
  if (dtype == 1) {
    if (WT) {  // k-contiguous blocks of 256 vocabulary entries
      const int T = dh_tile16(d);
      GemmGrid G{cdiv(d, T), cdiv(rows, kTile), nsplit, (int)k_split, (int)V_pad, 0, 0};
      Operand A{WT, 256, (int)d, (int)V_pad, d * 256};
      return run16(T, A, B, G, e, s);
    }
    GemmGrid G{cdiv(d, kTile), cdiv(rows, kTile), nsplit, (int)k_split, (int)V_pad, 0, 0};
    Operand A{W, d, (int)d, (int)V, 256};  // W itself, read transposed through LDS
    hipLaunchKernelGGL((gemm_pipe_kernel<OP_MC, OP_KC, EpiHeadDh, 2, 2, 64, 4, kTile>),
                       dim3((unsigned)(G.ntm * G.ntn * G.nsplit)), dim3(512), 0, s, A, B, G, e);
    return hipGetLastError();
  }
  Operand A{W, d, (int)d, (int)V, 256};
  return g32::run<OP_MC, OP_KC>(dh_tile32(C_alloc, d), d, rows, nsplit, k_split, V_pad, A, B, e, s);
}

// D[v][j] = sum_c dz[c][v] h[c][j] over k tokens (bf16: dzT and hT in blocks of 256 tokens)
hipError_t launch_head_dw(int dtype, int out, const void *dz, const void *dzt, const void *h_c,
                          const void *ht, int64_t k, int64_t d, int64_t V, int64_t V_pad,
                          int64_t C_alloc, const float *old, void *dW, hipStream_t s) {
  if (dtype == 1) {
    const int T = tile16(V, d);
    GemmGrid G{cdiv(V, T), cdiv(d, kTile), 1, (int)k, (int)k, 0, 0};
    Operand A{dzt, 256, (int)V, (int)k, V_pad * 256};
    Operand B{ht, 256, (int)d, (int)k, d * 256};
    if (out == 1) {
      EpiHeadDw<1> e{dW, old, (int)d, (int)V};
      return run16(T, A, B, G, e, s);
    }
    EpiHeadDw<0> e{dW, old, (int)d, (int)V};
    return run16(T, A, B, G, e, s);
  }
  Operand A{dz, 256, (int)V_pad, (int)k, C_alloc * 256};
  Operand B{h_c, d, (int)d, (int)k, 256};
  EpiHeadDw<0> e{dW, old, (int)d, (int)V};
  return g32::run<OP_MC, OP_MC>(g32::tile(V, d, 1), V, d, 1, k, k, A, B, e, s);
}

}  // namespace kd
