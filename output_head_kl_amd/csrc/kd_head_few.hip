// Log probabilities from hidden states of few tokens (a decoding step): z = h W^T where W is
// far larger than everything else, so the time is that of reading W once; and their gradients.
//
// A workgroup of four waves takes 64 or 128 vocabulary rows for all tokens (16 per MFMA column
// block, NC blocks).  W goes straight from memory into the registers of the matrix
// instructions, a ring of loads per wave in flight; the tokens' hidden states, read again by
// every workgroup but small and in L2, pass through LDS a chunk of k at a time: waiting for
// them (LDS counts apart) then does not wait for W.  The k order within a fragment is the
// memory's on both sides, which is all a dot product needs.  Per workgroup and token one
// (max, S = sum 2^t, sum t 2^t) partial, t = (z - max) log2 e, as in kd_head.hip.
// With one token of d 4096 over 128256 rows (1.05 GB) the call takes 198 us, 5.3 TB/s; 48 tokens
// of d 2880 over 201088 rows (1.16 GB) 245 us, 4.7 TB/s.  The GEMM tiles of more tokens are
// bound by W too there (64 tokens of d 4096 this way 226 us, 65 the other 229), but take longer
// where W is small (64 tokens, d 1024, V 32000: 22 us; 65: 34).
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

template <int DT, int NC> struct FewLds {
  static constexpr int CB = few_ring(NC) * 64, PITCH = CB + 16, TOK = 16 * NC;  // k bytes a chunk
  static constexpr int BYTES = 2 * TOK * PITCH;
};

// acc[r][n] += the product of the wave's rows v0 + 16 r .. and the tokens 16 n .. of h; lane l
// then holds token l % 16 and rows (l / 16) * 4 + i of a block.  hs: LDS, free afterwards.
template <int DT, int NC, int RB>
__device__ __forceinline__ void few_product(const char *W, const char *h, int rows, int d, int V,
                                            int v0, char *hs, f32x4 (&acc)[RB][NC]) {
  using L = FewLds<DT, NC>;
  constexpr int R = few_ring(NC), BURST = few_burst(NC), CB = L::CB;
  constexpr int HL = L::TOK * CB / 16 / kFewThreads;  // 16-byte pieces of h per thread and chunk
  static_assert(HL * kFewThreads * 16 == L::TOK * CB, "whole pieces");
  const int t = threadIdx.x, lane = t & 63;
  const int kb = d * FewT<DT>::ES, kl = kb - 16;  // bytes of a row (multiple of 16), last piece
  const int g16 = (lane >> 4) * 16;               // the lane group's place in 64 bytes of k
  const char *wp[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int v = v0 + r * 16 + (lane & 15);
    wp[r] = W + (long long)(v < V ? v : V - 1) * kb;  // the caller drops rows past V
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
      *(LDS_AS u32x4 *)((LDS_AS char *)hs + (buf * L::TOK + c) * L::PITCH + o) =
          k + o <= kl ? hr[i] : zero;
    }
  };
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
        const u32x4 b = *(const LDS_AS u32x4 *)((const LDS_AS char *)hs +
                                                (buf * L::TOK + n * 16 + (lane & 15)) * L::PITCH +
                                                s * 64 + g16);
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
}

template <int DT, int NC, int RB>
__global__ __launch_bounds__(kFewThreads) void k_head_few(const char *W, const char *h, int rows,
                                                          int d, int V, Tokens tokens,
                                                          float2 *part, float *part_t, float *zt) {
  constexpr int NW = kFewWaves, ROWS = NW * RB * 16, TOK = 16 * NC;
  __shared__ __attribute__((aligned(16))) char hs[FewLds<DT, NC>::BYTES];
  __shared__ float sp[NW][3][TOK];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int v0 = blockIdx.x * ROWS + w * RB * 16;
  f32x4 acc[RB][NC];
  few_product<DT, NC, RB>(W, h, rows, d, V, v0, hs, acc);

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

// Gradients of few tokens in bf16: z again, dz, and dW = dz^T h in one pass that reads W once
// and writes dW once; dz also goes out for the dh product.
//
// dz is kept as two bf16 numbers, hi + lo, side by side as twice as many tokens: the products
// then carry 16 bits of it, and dh and dW are rounded once in effect, where a single bf16 dz
// would leave the error of a few large elements in them (with one token up to 2^-9 of dW).  The
// matrix instructions have the room: all of this is bound by W and dW.
//
// After few_product a wave holds dz of its own 16 vocabulary rows for all tokens.  Through its
// own slice of LDS that becomes the B operand (k = token) of D[j][v].  A = hT, 64 hidden units
// a step, in chunks that the four waves share in LDS (fragments straight from L2 took twice the
// time: the pass then moves more of hT than of dW).  Row r of block b of A stands for hidden
// unit (b / 2) * 32 + (r / 4) * 8 + b % 2 * 4 + r % 4 for a bf16 dW, b * 16 + r for a float32
// one, so that a lane's accumulators are 16-byte pieces of rows of dW and four lanes write 64
// bytes side by side.  32 rows a wave were no faster (48 tokens, d 2880, V 201088: 867 us of
// gradients against 855), nor larger chunks.
struct FewBwd {
  const char *W, *h;
  const unsigned short *ht;  // (j, c) at j * 256 + c, zero for c >= rows
  int rows, d, V;
  Tokens tokens;
  LpGrad g;
  unsigned short *dz;        // null, or per 32 vocabulary rows [hi, lo][16 tokens][8 rows][16][8]
  void *dW;                  // null, or [V][d] of type OUT
  int stream;                // dW is larger than the last-level cache
};

template <int NC, int OUT>
__global__ __launch_bounds__(kFewThreads) void k_head_few_bwd(FewBwd a) {
  constexpr int NW = kFewWaves, ROWS = NW * 16, TOK = 16 * NC, K2 = 2 * TOK;
  constexpr int KS = K2 / 32, KA = TOK >= 32 ? TOK / 32 : 1;  // k-steps, different ones of hT
  constexpr int SP = K2 * 2 + 16, SLICES = NW * 16 * SP;
  constexpr int LDS = FewLds<1, NC>::BYTES > SLICES ? FewLds<1, NC>::BYTES : SLICES;
  __shared__ __attribute__((aligned(16))) char hs[LDS];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, g = lane >> 4;
  const int v0 = blockIdx.x * ROWS + w * 16;
  f32x4 acc[1][NC];
  few_product<1, NC, 1>(a.W, a.h, a.rows, a.d, a.V, v0, hs, acc);

  LDS_AS char *sl = (LDS_AS char *)hs + w * 16 * SP;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = n * 16 + (lane & 15);
    const bool cv = c < a.rows;
    const HeadTok k = cv ? head_tok(a.tokens, a.g, c, a.V) : HeadTok{0.f, 0.f, 0.f, 0.f, -1};
    unsigned short hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = v0 + g * 4 + i;
      const float q = fmaf(acc[0][n][i], kLog2e, -k.l2);  // log2 p
      float x = fmaf(fast_exp2(q), fmaf(k.b, q, k.a), v == k.tok ? k.g : 0.f);
      if (!cv || v >= a.V) x = 0.f;
      hi[i] = f32_to_bf16(x);
      lo[i] = f32_to_bf16(x - bf16_to_f32(hi[i]));
      LDS_AS char *at = sl + (g * 4 + i) * SP + c * 2;
      *(LDS_AS unsigned short *)at = hi[i];
      *(LDS_AS unsigned short *)(at + TOK * 2) = lo[i];
    }
    if (a.dz) {
      const int v = v0 + g * 4;
      unsigned short *to = a.dz + ((long long)(v >> 5) * 2 * NC + n) * 512 + (v >> 3 & 3) * 128 +
                           (lane & 15) * 8 + (v & 4);
      *(u32x2 *)to = u32x2{hi[0] | (unsigned)hi[1] << 16, hi[2] | (unsigned)hi[3] << 16};
      *(u32x2 *)(to + NC * 512) =
          u32x2{lo[0] | (unsigned)lo[1] << 16, lo[2] | (unsigned)lo[3] << 16};
    }
  }
  if (!a.dW) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the slice is the wave's own
  bf16x8 fb[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s)
    fb[s] = *(const LDS_AS bf16x8 *)(sl + (lane & 15) * SP + s * 64 + g * 16);

  // Chunks of JC hidden units in LDS as [block of 16][8 tokens][16 rows]: a fragment is read
  // without conflicts.  They are loaded two ahead, since a wait for a load is also one for the
  // stores before it.
  constexpr int PARTS = TOK / 8, HB = 8192, JC = HB / (TOK * 2), PP = HB / 16 / kFewThreads;
  u32x4 pre[2][PP];
  auto load_t = [&](u32x4 (&x)[PP], int j0) {
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int q = t + i * kFewThreads, j = j0 + q / PARTS;
      x[i] = *(const u32x4 *)(a.ht + (long long)(j < a.d ? j : a.d - 1) * 256 + q % PARTS * 8);
    }
  };
  auto store_t = [&](const u32x4 (&x)[PP], int buf) {
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int q = t + i * kFewThreads, j = q / PARTS;
      const int b = OUT == 1 ? (j >> 5) * 2 + (j >> 2 & 1) : j >> 4;
      const int r = OUT == 1 ? (j >> 3 & 3) * 4 + (j & 3) : j & 15;
      *(LDS_AS u32x4 *)((LDS_AS char *)hs + buf * HB + ((b * PARTS + q % PARTS) * 16 + r) * 16) =
          x[i];
    }
  };
  auto chunk = [&](int jc, int buf) {
#pragma unroll 1
    for (int jj = 0; jj < JC && jc + jj < a.d; jj += 64) {
      bf16x8 fa[4][KA];
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int s = 0; s < KA; ++s)
          fa[b][s] = *(const LDS_AS bf16x8 *)((LDS_AS char *)hs + buf * HB +
                                              ((((jj >> 4) + b) * PARTS + (s * 4 + g) % PARTS) *
                                                   16 + (lane & 15)) * 16);
      f32x4 o[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        o[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
          o[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[b][s % KA], fb[s], o[b], 0, 0, 0);
      }
      const int v = v0 + (lane & 15);
      if (v >= a.V) continue;
#pragma unroll
      for (int q = 0; q < (OUT == 1 ? 2 : 4); ++q) {
        const int j = jc + jj + (OUT == 1 ? q * 32 + g * 8 : q * 16 + g * 4);
        if (j >= a.d) break;  // d is a multiple of 8
        const long long e = (long long)v * a.d + j;
        u32x4 x, *to;
        if (OUT == 1) {
          const f32x4 x0 = o[2 * q % 4], x1 = o[(2 * q + 1) % 4];
          x = u32x4{pack_bf16x2(x0[0], x0[1]), pack_bf16x2(x0[2], x0[3]),
                    pack_bf16x2(x1[0], x1[1]), pack_bf16x2(x1[2], x1[3])};
          to = (u32x4 *)((unsigned short *)a.dW + e);
        } else {
          x = __builtin_bit_cast(u32x4, o[q]);
          to = (u32x4 *)((float *)a.dW + e);
        }
        if (a.stream) __builtin_nontemporal_store(x, to);
        else *to = x;
      }
    }
  };
  load_t(pre[0], 0);
  load_t(pre[1], JC);
  few_sync();  // every wave has read its slice
  store_t(pre[0], 0);
  load_t(pre[0], 2 * JC);
  few_sync();
  for (int jc = 0; jc < a.d; jc += 2 * JC) {
    chunk(jc, 0);
    store_t(pre[1], 1);
    load_t(pre[1], jc + 3 * JC);
    few_sync();
    chunk(jc + JC, 1);
    store_t(pre[0], 0);
    load_t(pre[0], jc + 4 * JC);
    few_sync();
  }
}

// dh = dz W of few tokens: D[j][c] = sum_v W[v][j] (hi + lo)[c][v], W read once.
//
// The sum's index is W's row, so a lane loads 16 bytes (8 hidden units) of 8 rows and turns them
// by byte permutations, 32 for 64 elements: register p of the fragment for unit jj holds rows 2p
// and 2p + 1.  Row m of fragment jj is unit 8 m + jj, 16 lanes read 256 bytes of a row, and a
// lane's results are 8 neighbouring units.  hi and lo add to the same accumulators.  A wave has
// 128 units and the four waves of a workgroup share dz through LDS; the rows of W are split
// over about one workgroup a CU (two a CU, with twice the partial sums: 40 us longer), whose
// partial sums k_head_few_dh_join adds in order.
constexpr int kFewDhGroups = 256;
template <int NC>
__global__ __launch_bounds__(kFewThreads) void k_head_few_dh(const char *W,
                                                             const unsigned short *dz, int d,
                                                             int V, int k_split, int v_end,
                                                             float *part, int d_pad) {
  constexpr int TOK = 16 * NC, KC = 8 / NC, STEP = 2 * NC * 1024;
  constexpr int CB = KC * STEP, PZ = CB / 16 / kFewThreads;
  __shared__ __attribute__((aligned(16))) char hs[2 * CB];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, g = lane >> 4;
  
  // the workgroups of a split share dz: on one XCD (workgroups go round the eight of them)
  const int tiles = (d + kFewWaves * 128 - 1) / (kFewWaves * 128), slot = blockIdx.x >> 3;
  const int split = (slot / tiles) * 8 + (blockIdx.x & 7), k0 = split * k_split;
  if (k0 >= v_end) return;
  const int k1 = k0 + k_split < v_end ? k0 + k_split : v_end;  // whole chunks of KC * 32 rows
  const int j0 = (slot % tiles * kFewWaves + w) * 128, ja = j0 + (lane & 15) * 8;
  const unsigned short *wj = (const unsigned short *)W + (ja < d ? ja : d - 8);
  u32x4 wr[2][8], pre[PZ];
  auto load_w = [&](u32x4 (&x)[8], int k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int v = k + g * 8 + i;  // past V dz is zero
      x[i] = *(const u32x4 *)(wj + (long long)(v < V ? v : V - 1) * d);
    }
  };
  auto load_z = [&](int k) {
#pragma unroll
    for (int i = 0; i < PZ; ++i)
      pre[i] = *(const u32x4 *)((const char *)dz + (long long)((k < k1 ? k : k0) >> 5) * STEP +
                                (t + i * kFewThreads) * 16);
  };
  auto store_z = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PZ; ++i)
      *(LDS_AS u32x4 *)((LDS_AS char *)hs + buf * CB + (t + i * kFewThreads) * 16) = pre[i];
  };
  f32x4 acc[8][NC];
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int n = 0; n < NC; ++n) acc[q][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  load_z(k0);
#pragma unroll
  for (int u = 0; u < 2; ++u) load_w(wr[u], k0 + u * 32);
  store_z(0);
  few_sync();
  int buf = 0;
  for (int k = k0; k < k1; k += KC * 32, buf ^= 1) {
    load_z(k + KC * 32);
#pragma unroll 1
    for (int s = 0; s < KC; s += 2)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        bf16x8 fb[2][NC];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int n = 0; n < NC; ++n)
            fb[x][n] = *(const LDS_AS bf16x8 *)((const LDS_AS char *)hs + buf * CB +
                                                (s + u) * STEP + (x * NC + n) * 1024 + lane * 16);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          u32x4 fa;
#pragma unroll
          for (int p = 0; p < 4; ++p)
            fa[p] = __builtin_amdgcn_perm(wr[u][2 * p + 1][q / 2], wr[u][2 * p][q / 2],
                                          q & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int n = 0; n < NC; ++n)
              acc[q][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, fa), fb[x][n], acc[q][n], 0, 0, 0);
        }
        load_w(wr[u], k + (s + u + 2) * 32);
        __builtin_amdgcn_sched_barrier(0);
      }
    store_z(buf ^ 1);
    few_sync();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + (g * 4 + i) * 8;
    if (j >= d_pad) continue;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      float *to = part + ((long long)split * TOK + n * 16 + (lane & 15)) * d_pad + j;
      *(f32x4 *)to = f32x4{acc[0][n][i], acc[1][n][i], acc[2][n][i], acc[3][n][i]};
      *(f32x4 *)(to + 4) = f32x4{acc[4][n][i], acc[5][n][i], acc[6][n][i], acc[7][n][i]};
    }
  }
}

// dh[c][j] = the splits' sum, rounded once: four units a thread, each quarter of a workgroup a
// quarter of the splits.
__global__ __launch_bounds__(256) void k_head_few_dh_join(const float *part, int nsplit, int tok,
                                                          int d_pad, int rows, int d,
                                                          unsigned short *dh) {
  __shared__ f32x4 sx[3][64];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int q = d / 4, i = blockIdx.x * 64 + lane;
  const int c = i / q, j = (i - c * q) * 4;
  const int s0 = nsplit * w / 4, s1 = nsplit * (w + 1) / 4;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if (i < rows * q) {
#pragma unroll 8
    for (int s = s0; s < s1; ++s)
      x += *(const f32x4 *)(part + ((long long)s * tok + c) * d_pad + j);
  }
  if (w) sx[w - 1][lane] = x;
  __syncthreads();
  if (w || i >= rows * q) return;
  x = (x + sx[0][lane]) + (sx[1][lane] + sx[2][lane]);
  *(u32x2 *)(dh + (long long)c * d + j) =
      u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
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

namespace {
template <int OUT>
void run_head_few_bwd(const FewBwd &a, int64_t V_pad, hipStream_t s) {
  const int tok = head_few_tokens(a.rows);
  const dim3 grid((unsigned)(V_pad / (kFewWaves * 16))), block(kFewThreads);
#define KD_FEW(NC) hipLaunchKernelGGL((k_head_few_bwd<NC, OUT>), grid, block, 0, s, a)
  if (tok == 16) KD_FEW(1);
  else if (tok == 32) KD_FEW(2);
  else KD_FEW(4);
#undef KD_FEW
}
}  // namespace

int head_few_dh_splits(int64_t d, int64_t V) {
  const int64_t tiles = cdiv(d, kFewWaves * 128), most = cdiv(V, 256);
  const int64_t n = kFewDhGroups / tiles / 8 * 8;
  return (int)(n < 8 ? most < 8 ? most : 8 : n < most ? n : most);
}

hipError_t launch_head_few_bwd(const void *W, const void *h, const void *ht, int64_t rows,
                               int64_t d, int64_t V, int64_t V_pad, const Tokens &tokens,
                               const LpGrad &g, void *dz, void *dW, int out, hipStream_t s) {
  const FewBwd a{(const char *)W, (const char *)h, (const unsigned short *)ht, (int)rows, (int)d,
                 (int)V, tokens, g, (unsigned short *)dz, dW,
                 V * d * (out == 1 ? 2 : 4) > ((int64_t)256 << 20)};
  if (out == 1) run_head_few_bwd<1>(a, V_pad, s);
  else run_head_few_bwd<0>(a, V_pad, s);
  return hipGetLastError();
}

hipError_t launch_head_few_dh(const void *W, const void *dz, int64_t rows, int64_t d, int64_t V,
                              int64_t V_pad, int nsplit, float *part, void *dh, hipStream_t s) {
  const int tok = head_few_tokens(rows), d_pad = (int)((d + 127) / 128 * 128);
  const int64_t k_split = cdiv(cdiv(V_pad, 256), nsplit) * 256, used = cdiv(V_pad, k_split);
  const dim3 grid(cdiv(d, kFewWaves * 128) * cdiv(used, 8) * 8), block(kFewThreads);
#define KD_FEW(NC)                                                                              \
  hipLaunchKernelGGL((k_head_few_dh<NC>), grid, block, 0, s, (const char *)W,                   \
                     (const unsigned short *)dz, (int)d, (int)V, (int)k_split, (int)V_pad, part, \
                     d_pad)
  if (tok == 16) KD_FEW(1);
  else if (tok == 32) KD_FEW(2);
  else KD_FEW(4);
#undef KD_FEW
  hipLaunchKernelGGL(k_head_few_dh_join, dim3(cdiv(rows * (d / 4), 64)), dim3(256), 0, s, part,
                     (int)used, tok, d_pad, (int)rows, (int)d, (unsigned short *)dh);
  return hipGetLastError();
}

}  // namespace kd
