// float32 MFMA GEMM on tiles of 128 x 128 or 64 x 64, for the log probabilities from float32
// hidden states.
//
// D[m][n] = sum_k A[m][k] B[k][n], operands and epilogues as in kd_gemm.h.  Four waves of T/2 x
// T/2 (one or two by two blocks of the 32x32x2 MFMA, 64 cycles each), k in steps of 32, two LDS
// stages filled through registers: bound by the matrix instructions.  The next stage's loads go
// out before a step's products and reach LDS half-way through them, fragments are read one
// eighth of k ahead.  4096 tokens, d 1024, V 32000 run at 123 TFLOP/s forward and 120 over the
// three products of the gradients (a library's plain product of that shape at 140, the 256 x
// 256 tile of kd_gemm.h at 121), but small shapes fill the chip: 512 tokens, d 256, V 8192 take
// 29 us forward instead of 84.
#pragma once

#include "kd_gemm.h"

namespace kd {
namespace g32 {

constexpr int BK = 32;
// KC: [T rows][128 B], 16-byte chunks swizzled by row so that 16 rows' chunks of a fragment fall
// on all 64 banks; MC: [32 k][T mn], padded rows
template <int T> constexpr int mc_pitch() { return T * 4 + 16; }
template <int T, int KIND> constexpr int bytes() {
  return KIND == OP_KC ? T * BK * 4 : BK * mc_pitch<T>();
}
// The tile with less work on the fullest compute unit, in 64 x 64 tiles: those run 8 % slower
// per element (2048 tokens, d 512, V 8192 forward: 161 against 149 us) but fill the chip more
// evenly (1203 tokens, d 2680, V 8047: 493 against 546 us), and a lone large one waits more.
inline int tile(int64_t m, int64_t n, int64_t splits) {
  auto fullest = [&](int64_t t) { return ((m + t - 1) / t * ((n + t - 1) / t) * splits + 255) / 256; };
  const double large = 4.0 * (double)fullest(128) * (fullest(128) == 1 ? 1.1 : 1.0);
  return 1.08 * (double)fullest(64) < large ? 64 : 128;
}

// Chunk q = t + 256 i of a stage: (mn, k) and its place in LDS.
template <int T, int KIND>
__device__ __forceinline__ void chunk(int q, int &mn, int &k, int &at) {
  if (KIND == OP_KC) {
    mn = q >> 3;
    k = (q & 7) * 4;
    at = mn * 128 + (((q & 7) ^ (mn >> 1 & 7)) << 4);
  } else {
    k = q / (T / 4);
    mn = (q % (T / 4)) * 4;
    at = k * mc_pitch<T>() + mn * 4;
  }
}

// k and mn extents are multiples of 4 in the contiguous direction, so a chunk is inside or not.
// One outside is loaded from the last place inside and becomes zero on its way to LDS: a load
// under a condition would be waited for at once.
template <int T, int KIND>
__device__ __forceinline__ void load(u32x4 (&r)[T / 32], const Operand &op, int mn0, int k0, int t) {
  const int last_mn = op.mn_ext - (KIND == OP_KC ? 1 : 4), last_k = op.k_ext - (KIND == OP_KC ? 4 : 1);
#pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    int mn, k, at;
    chunk<T, KIND>(t + 256 * i, mn, k, at);
    r[i] = *(const u32x4 *)((const float *)op.ptr +
                            op_index(op, KIND, min(mn + mn0, last_mn), min(k + k0, last_k)));
  }
}

template <int T, int KIND>
__device__ __forceinline__ void store(char *lds, const u32x4 (&r)[T / 32], const Operand &op,
                                      int mn0, int k0, int t) {
#pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    int mn, k, at;
    chunk<T, KIND>(t + 256 * i, mn, k, at);
    const u32x4 zero = {0u, 0u, 0u, 0u};
    *(LDS_AS u32x4 *)((LDS_AS char *)lds + at) =
        mn + mn0 < op.mn_ext && k + k0 < op.k_ext ? r[i] : zero;
  }
}

// Rows r0 .. r0 + 31, k-substep ks (8 of k): lane l holds row l % 32, k 4 (l / 32) .. + 3.
template <int T, int KIND>
__device__ __forceinline__ f32x4 frag(const char *lds, int r0, int ks, int lane) {
  const LDS_AS char *b = (const LDS_AS char *)lds;
  const int row = r0 + (lane & 31);
  if (KIND == OP_KC) {
    const int kc = ks * 2 + (lane >> 5);
    return *(const LDS_AS f32x4 *)(b + row * 128 + ((kc ^ (row >> 1 & 7)) << 4));
  }
  const int k = ks * 8 + (lane >> 5) * 4;
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = *(const LDS_AS float *)(b + (k + e) * mc_pitch<T>() + row * 4);
  return v;
}

template <int T, int AK, int BKIND, class Epi>
__global__ __launch_bounds__(256, 2) void gemm32_kernel(Operand A, Operand B, GemmGrid G, Epi epi) {
  constexpr int AB = bytes<T, AK>(), STAGE = AB + bytes<T, BKIND>(), NB = T / 64;
  __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];
  const int lin = xcd_remap(blockIdx.x, gridDim.x);
  const int per_split = G.ntm * G.ntn, split = lin / per_split, rem = lin - split * per_split;
  const int tm = rem / G.ntn, tn = rem - tm * G.ntn;
  const int m0 = tm * T, n0 = tn * T;
  const int kb = split * G.k_len, ke = min(G.k_total, kb + G.k_len);
  const int nk = ke > kb ? (ke - kb + BK - 1) / BK : 0;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, wr = w >> 1, wc = w & 1;
  A.k_ext = min(A.k_ext, ke);
  B.k_ext = min(B.k_ext, ke);
  f32x16 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
  u32x4 ra[T / 32], rb[T / 32];
  load<T, AK>(ra, A, m0, kb, t);
  load<T, BKIND>(rb, B, n0, kb, t);
  store<T, AK>(smem, ra, A, m0, kb, t);
  store<T, BKIND>(smem + AB, rb, B, n0, kb, t);
  __syncthreads();
  for (int it = 0; it < nk; ++it) {
    const int k1 = kb + (it + 1) * BK;
    load<T, AK>(ra, A, m0, k1, t);  // past the last step: loaded, not stored
    load<T, BKIND>(rb, B, n0, k1, t);
    __builtin_amdgcn_sched_barrier(0);  // the loads go out before the step's products
    const char *la = smem + (it & 1) * STAGE, *lb = la + AB;
    f32x4 fa[2][NB], fb[2][NB];
    auto frags = [&](int ks) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
        fa[ks & 1][i] = frag<T, AK>(la, wr * (T / 2) + i * 32, ks, lane);
#pragma unroll
      for (int j = 0; j < NB; ++j)
        fb[ks & 1][j] = frag<T, BKIND>(lb, wc * (T / 2) + j * 32, ks, lane);
    };
    frags(0);
#pragma unroll
    for (int ks = 0; ks < BK / 8; ++ks) {
      if (ks + 1 < BK / 8) frags(ks + 1);
      if (ks == BK / 16 && it + 1 < nk) {  // between products, so they cover its waits
        char *nxt = smem + ((it + 1) & 1) * STAGE;
        store<T, AK>(nxt, ra, A, m0, k1, t);
        store<T, BKIND>(nxt + AB, rb, B, n0, k1, t);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = mma(fa[ks & 1][i], fb[ks & 1][j], acc[i][j]);
    }
    __syncthreads();
  }
  epi(acc, m0 + wr * (T / 2), n0 + wc * (T / 2), lane, split, smem);
}

// m x n outputs on T x T tiles (T 64 or 128).
template <int AK, int BKIND, class Epi>
static hipError_t run(int T, int64_t m, int64_t n, int nsplit, int64_t k_len, int64_t k_total,
                      const Operand &A, const Operand &B, const Epi &epi, hipStream_t s) {
  const GemmGrid G{cdiv(m, T), cdiv(n, T), nsplit, (int)k_len, (int)k_total, 0, 0};
  const dim3 grid((unsigned)((long long)G.ntm * G.ntn * nsplit)), block(256);
  if (T == 64)
    hipLaunchKernelGGL((gemm32_kernel<64, AK, BKIND, Epi>), grid, block, 0, s, A, B, G, epi);
  else
    hipLaunchKernelGGL((gemm32_kernel<128, AK, BKIND, Epi>), grid, block, 0, s, A, B, G, epi);
  return hipGetLastError();
}

}  // namespace g32
}  // namespace kd
