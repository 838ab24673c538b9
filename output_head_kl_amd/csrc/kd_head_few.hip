// Log probabilities from hidden states of few tokens (a decoding step): z = h W^T where W is
// far larger than everything else, so the time is that of reading W once.
//
// A workgroup of four waves takes 64 or 128 vocabulary rows for all tokens (16 per MFMA column
// block, NC blocks).  W goes straight from memory into the registers of the matrix
// instructions, a ring of loads per wave in flight; the tokens' hidden states, read again by
// every workgroup but small and in L2, pass through LDS a chunk of k at a time: waiting for
// them (LDS counts apart) then does not wait for W.  The k order within a fragment is the
// memory's on both sides, which is all a dot product needs.  Per workgroup and token one
// (max, S = sum 2^t, sum t 2^t) partial, t = (z - max) log2 e, as in kd_head.hip.
// With one token of d 4096 over 128256 rows (1.05 GB) the call takes 194 us, 5.4 TB/s; the
// 256-column GEMM tile takes 306 us there and 335 us for 48 tokens of d 2880 over 201088 rows.
// W through an LDS ring instead (loads of whole lines straight into it) measured 215 and 273 us,
// non-temporal loads of W 212 and 302 us (a line's second half is then fetched twice).
#include "kd_gemm.h"
#include "kd_ops.h"

namespace kd {
namespace {

template <int DT> struct FewT;
template <> struct FewT<1> { static constexpr int ES = 2; };
template <> struct FewT<0> { static constexpr int ES = 4; };

// acc += A B over the 64 bytes of k (per row and per token) that the four lane groups hold
// 16 bytes each of.
template <int DT>
__device__ __forceinline__ f32x4 few_mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == 1) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0,
                                               0, 0);
    return c;
  }
}

// Barrier for LDS alone: the loads of W stay in flight.
__device__ __forceinline__ void few_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A wave's rows (RB blocks of 16) and its ring of R loads of 64 bytes of k per row.  Up to 16
// tokens: 16 rows and a ring of eight, renewed load by load.  More: 32 rows, which halve what
// is read of h per byte of W, and a ring of four renewed at once, so that a row's 256 bytes are
// asked for together (201088 x 2880, 48 tokens: 250 us; renewed load by load 280; 16 rows 262;
// eight deep 263 and 291), unless the vocabulary is too small to give every compute unit two
// workgroups of such rows (14000 x 512, 64 tokens: 12.4 us with 16 rows, 15.5 with 32).
constexpr int kFewWaves = 4, kFewThreads = 64 * kFewWaves;
constexpr int few_ring(int nc) { return nc == 1 ? 8 : 4; }
constexpr int few_burst(int nc) { return nc == 1 ? 1 : 4; }
inline int few_blocks(int64_t N, int64_t V) { return N <= 16 || V < 65536 ? 1 : 2; }

template <int DT, int NC, int RB>
__global__ __launch_bounds__(kFewThreads) void k_head_few(const char *W, const char *h, int rows,
                                                          int d, int V, Tokens tokens,
                                                          float2 *part, float *part_t, float *zt) {
  constexpr int ES = FewT<DT>::ES, R = few_ring(NC), BURST = few_burst(NC), NW = kFewWaves;
  constexpr int ROWS = NW * RB * 16;
  constexpr int CB = R * 64, PITCH = CB + 16, TOK = 16 * NC;  // bytes of k a chunk
  constexpr int HL = TOK * CB / 16 / kFewThreads;  // 16-byte pieces of h per thread and chunk
  static_assert(HL * kFewThreads * 16 == TOK * CB, "whole pieces");
  __shared__ __attribute__((aligned(16))) char hs[2][TOK * PITCH];
  __shared__ float sp[NW][3][TOK];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int v0 = blockIdx.x * ROWS + w * RB * 16;
  const int kb = d * ES, kl = kb - 16;  // bytes of a row, a multiple of 16, and its last piece
  const int g16 = (lane >> 4) * 16;     // the lane group's place in 64 bytes of k
  const char *wp[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int v = v0 + r * 16 + (lane & 15);
    wp[r] = W + (long long)(v < V ? v : V - 1) * kb;  // rows past V are dropped at the end
  }
  // 16 bytes at k (bytes) of a row.  Past its end the row's last 16 bytes are loaded again, and
  // meet zeros of h: no load is conditional (each would be waited for at once).
  auto load_w = [&](int r, int k) {
    return *(const u32x4 *)(wp[r] + (k + g16 < kl ? k + g16 : kl));
  };
  u32x4 hr[HL];
  auto load_h = [&](int k) {
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      const int q = t + i * kFewThreads, c = q / (CB / 16), o = k + (q % (CB / 16)) * 16;
      hr[i] = *(const u32x4 *)(h + (long long)(c < rows ? c : rows - 1) * kb + (o < kl ? o : kl));
    }
  };
  auto store_h = [&](int buf, int k) {
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      const int q = t + i * kFewThreads, c = q / (CB / 16), o = (q % (CB / 16)) * 16;
      const u32x4 zero = {0u, 0u, 0u, 0u};
      *(LDS_AS u32x4 *)((LDS_AS char *)hs[buf] + c * PITCH + o) = k + o <= kl ? hr[i] : zero;
    }
  };
  f32x4 acc[RB][NC];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int n = 0; n < NC; ++n) acc[r][n] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 a[R][RB];
  load_h(0);
#pragma unroll
  for (int s = 0; s < R; ++s)
#pragma unroll
    for (int r = 0; r < RB; ++r) a[s][r] = load_w(r, s * 64);
  store_h(0, 0);
  few_sync();
  int buf = 0;
  for (int k = 0; k < kb; k += CB, buf ^= 1) {
    load_h(k + CB);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < R; ++s) {
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const u32x4 b = *(const LDS_AS u32x4 *)((const LDS_AS char *)hs[buf] +
                                                (n * 16 + (lane & 15)) * PITCH + s * 64 + g16);
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[r][n] = few_mma<DT>(a[s][r], b, acc[r][n]);
      }
      if ((s + 1) % BURST == 0)
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
          for (int q = s + 1 - BURST; q <= s; ++q) a[q][r] = load_w(r, k + CB + q * 64);
      __builtin_amdgcn_sched_barrier(0);  // a step's loads are issued before the next waits
    }
    store_h(buf ^ 1, k + CB);
    few_sync();
  }

  // lane: token n * 16 + lane % 16, rows r * 16 + (lane / 16) * 4 + i
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = n * 16 + (lane & 15);
    const long long tok = c < rows ? tokens.at(c) : -1;
    float mx = -INFINITY;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = v0 + r * 16 + (lane >> 4) * 4 + i;
        if (v < V) {
          mx = fmaxf(mx, acc[r][n][i]);
          if (v == tok) zt[c] = acc[r][n][i];
        }
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    const float mx2 = mx * kLog2e;
    float s = 0.f, t2 = 0.f;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v0 + r * 16 + (lane >> 4) * 4 + i < V) {
          const float x = fmaf(acc[r][n][i], kLog2e, -mx2), e = fast_exp2(x);
          s += e;
          t2 = fmaf(e, x, t2);
        }
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    t2 += __shfl_xor(t2, 16, 64);
    t2 += __shfl_xor(t2, 32, 64);
    if (lane < 16) {
      sp[w][0][c] = mx;
      sp[w][1][c] = s;
      sp[w][2][c] = t2;
    }
  }
  __syncthreads();
  if (t >= TOK || t >= rows) return;
  // the four waves' partials of a token; a wave wholly past V has max -inf and adds nothing
  float M = sp[0][0][t];
#pragma unroll
  for (int i = 1; i < NW; ++i) M = fmaxf(M, sp[i][0][t]);
  float S = 0.f, T = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i)
    if (blockIdx.x * ROWS + i * RB * 16 < V) {
      const float x = fmaxf((sp[i][0][t] - M) * kLog2e, kOpLowest), c = fast_exp2(x);
      S = fmaf(c, sp[i][1][t], S);
      T = fmaf(c, fmaf(x, sp[i][1][t], sp[i][2][t]), T);
    }
  part[(long long)t * gridDim.x + blockIdx.x] = make_float2(M, S);
  part_t[(long long)t * gridDim.x + blockIdx.x] = T;
}

}  // namespace

int64_t head_few_partials(int64_t N, int64_t V) {
  const int rows = kFewWaves * 16 * few_blocks(N, V);
  return (V + rows - 1) / rows;
}

namespace {
template <int DT>
void run_head_few(dim3 grid, hipStream_t s, const char *W, const char *h, int rows, int d, int V,
                  const Tokens &tokens, float2 *part, float *part_t, float *zt) {
  const dim3 block(kFewThreads);
#define KD_FEW(NC, RB)                                                                         \
  hipLaunchKernelGGL((k_head_few<DT, NC, RB>), grid, block, 0, s, W, h, rows, d, V, tokens, part, \
                     part_t, zt)
  const bool two = few_blocks(rows, V) == 2;
  if (rows <= 16) KD_FEW(1, 1);
  else if (rows <= 32 && two) KD_FEW(2, 2);
  else if (rows <= 32) KD_FEW(2, 1);
  else if (two) KD_FEW(4, 2);
  else KD_FEW(4, 1);
#undef KD_FEW
}
}  // namespace

hipError_t launch_head_few(int dtype, const void *W, const void *h, int64_t rows, int64_t d,
                           int64_t V, const Tokens &tokens, float2 *part, float *part_t,
                           float *zt, hipStream_t s) {
  (dtype == 1 ? run_head_few<1> : run_head_few<0>)(
      dim3((unsigned)head_few_partials(rows, V)), s, (const char *)W, (const char *)h, (int)rows,
      (int)d, (int)V, tokens, part, part_t, zt);
  return hipGetLastError();
}

}  // namespace kd
