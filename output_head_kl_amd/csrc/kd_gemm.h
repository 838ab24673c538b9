// The MFMA GEMM core that the output-head kernels share: operand descriptions, the simple
// register-staged kernel (fp32), the pipelined bf16 kernel, and run_gemm, which launches
// the one that fits the element type with a caller-given epilogue.
#pragma once

#include "kd_internal.h"

#include <cstdint>
#include <type_traits>

namespace kd {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

#define LDS_AS __attribute__((address_space(3)))

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------------
// small helpers
// ---------------------------------------------------------------------------------
__device__ __forceinline__ float bf16_to_f32(unsigned short b) {
  return __uint_as_float(((unsigned int)b) << 16);
}
// Round to nearest, ties to even: gfx950's v_cvt_pk_bf16_f32 converts two floats in one
// instruction.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned int pack_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(unsigned int, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}
__device__ __forceinline__ unsigned short f32_to_bf16(float f) {
  return (unsigned short)(pack_bf16x2(f, 0.f) & 0xFFFFu);
}
__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Lanes l and l^32 hold the two halves of a token's values; combine them.
__device__ __forceinline__ float halves_max(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}
__device__ __forceinline__ double wave_sum_d(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// Workgroups are dispatched round-robin over the 8 XCDs (bid % 8).  Give each XCD a
// contiguous range of tile ids so that tiles sharing operands share that XCD's L2.
__device__ __forceinline__ int xcd_remap(int bid, int T) {
  const int q = T >> 3, r = T & 7, x = bid & 7, j = bid >> 3;
  return x * q + (x < r ? x : r) + j;
}

// ---------------------------------------------------------------------------------
// MFMA GEMM core
//
// D[m][n] = sum_k A[m][k] * B[k][n] over one 256 x 256 tile, K in steps of one
// 128-byte row chunk per operand row (64 bf16 or 32 fp32).  An operand is either
//   KC: stored [mn][k] (k contiguous) -> LDS [256 rows][128 B], 16-B chunks XOR
//       swizzled by row, fragments read with ds_read_b128;
//   MC: stored [k][mn] (mn contiguous) -> LDS [k rows][256 mn] padded rows,
//       fragments read transposed (ds_read_b64_tr_b16 for bf16).
// Each wave owns 128 x 128 of the tile as 4 x 4 blocks of the 32x32 MFMA;
// accumulator element i of lane l in block (rb, cb) is row
// rb*32 + (i/4)*8 + (l/32)*4 + i%4 and column cb*32 + l%32 of the wave's square.
// ---------------------------------------------------------------------------------
enum { OP_KC = 0, OP_MC = 1 };

// Element (mn, k) of an operand lives at
//   KC: ptr[(k / 256) * ts + k % 256 + mn * ld],  MC: ptr[(mn / 256) * ts + mn % 256 + k * ld].
// A plain row-major matrix has ts = 256; a matrix stored as blocks of 256 contiguous
// columns (each block [rows][256]) has ld = 256 and ts = rows * 256.
struct Operand {
  const void *ptr;
  long long ld;     // elements between rows
  int mn_ext;       // rows/cols with mn >= mn_ext read as zero
  int k_ext;        // k >= k_ext read as zero
  long long ts;     // elements between 256-column blocks
};

__device__ __forceinline__ long long op_index(const Operand &op, int kind, int mn, int k) {
  return kind == 0 ? (long long)(k >> 8) * op.ts + (k & 255) + (long long)mn * op.ld
                   : (long long)(mn >> 8) * op.ts + (mn & 255) + (long long)k * op.ld;
}

struct GemmGrid {
  int ntm, ntn, nsplit;
  int k_len;    // k range of one split (multiple of the k-step)
  int k_total;  // loop bound
  int order;    // 0: n-tile index fastest, 1: m-tile index fastest
  int ngrp;     // order 0 (bf16 pipe kernel): n tiles taken in groups of ngrp, all m
                // tiles of a group before the next group (0: one group)
};

template <int DT> struct Elem;
template <> struct Elem<1> {  // bf16
  static constexpr int CH = 8, BK = 64, ES = 2, MC_PITCH = 576, MC_ROWS = 64;
};
template <> struct Elem<0> {  // fp32
  static constexpr int CH = 4, BK = 32, ES = 4, MC_PITCH = 1088, MC_ROWS = 32;
};

template <int DT, int KIND> struct OpLds {
  static constexpr int BYTES = KIND == OP_KC ? 256 * 128 : Elem<DT>::MC_ROWS * Elem<DT>::MC_PITCH;
};

template <int DT, int KIND>
__device__ __forceinline__ void load_stage(u32x4 (&r)[8], const Operand &op, int mn0, int k0,
                                           int t) {
  constexpr int CH = Elem<DT>::CH, ES = Elem<DT>::ES;
  const char *base = (const char *)op.ptr;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = t + 256 * i;
    int mn, k;
    if (KIND == OP_KC) {
      mn = mn0 + (q >> 3);
      k = k0 + (q & 7) * CH;
    } else if (DT == 1) {
      k = k0 + (q >> 5);
      mn = mn0 + (q & 31) * CH;
    } else {
      k = k0 + (q >> 6);
      mn = mn0 + (q & 63) * CH;
    }
    const bool ok = mn < op.mn_ext && k < op.k_ext;
    const long long e = op_index(op, KIND, mn, k);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (ok) v = *(const u32x4 *)(base + e * ES);
    r[i] = v;
  }
}

template <int DT, int KIND>
__device__ __forceinline__ void store_stage(char *lds, const u32x4 (&r)[8], int t) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = t + 256 * i;
    int off;
    if (KIND == OP_KC) {
      const int row = q >> 3, kc = q & 7;
      off = row * 128 + ((kc ^ (row & 7)) << 4);
    } else if (DT == 1) {
      off = (q >> 5) * Elem<1>::MC_PITCH + (q & 31) * 16;
    } else {
      off = (q >> 6) * Elem<0>::MC_PITCH + (q & 63) * 16;
    }
    *(LDS_AS u32x4 *)((LDS_AS char *)lds + off) = r[i];
  }
}

// Fragment of 32 rows r0..r0+31 for k-substep ks (16 bf16 or 8 fp32 of k).
template <int DT, int KIND> struct Frag;

template <> struct Frag<1, OP_KC> {
  typedef bf16x8 type;
  static __device__ __forceinline__ type load(const char *lds, int r0, int ks, int lane) {
    const int row = r0 + (lane & 31), kc = ks * 2 + (lane >> 5);
    return *(const LDS_AS bf16x8 *)((const LDS_AS char *)lds + row * 128 + ((kc ^ (row & 7)) << 4));
  }
};
template <> struct Frag<1, OP_MC> {
  typedef bf16x8 type;
  // ds_read_b64_tr_b16: in each 16-lane group, lane j receives element j%4 of the
  // 8 bytes loaded by lanes j/4 + 4r, r = 0..3.  Lane s of the group loads the 4
  // values at [k = kb + s/4][m = mb + 4*(s%4) ..], so lane j gets [kb..kb+3][mb + j].
  static __device__ __forceinline__ type load(const char *lds, int r0, int ks, int lane) {
    const int s = lane & 15, g = lane >> 4;
    const int m = r0 + (g & 1) * 16 + 4 * (s & 3);
    const int k = ks * 16 + (g >> 1) * 8 + (s >> 2);
    const LDS_AS char *b = (const LDS_AS char *)lds;
    s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (LDS_AS s16x4 *)(b + k * Elem<1>::MC_PITCH + m * 2));
    s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (LDS_AS s16x4 *)(b + (k + 4) * Elem<1>::MC_PITCH + m * 2));
    s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
  }
};
template <> struct Frag<0, OP_KC> {
  typedef f32x4 type;
  static __device__ __forceinline__ type load(const char *lds, int r0, int ks, int lane) {
    const int row = r0 + (lane & 31), kc = ks * 2 + (lane >> 5);
    return *(const LDS_AS f32x4 *)((const LDS_AS char *)lds + row * 128 + ((kc ^ (row & 7)) << 4));
  }
};
template <> struct Frag<0, OP_MC> {
  typedef f32x4 type;
  static __device__ __forceinline__ type load(const char *lds, int r0, int ks, int lane) {
    const int m = r0 + (lane & 31), k = ks * 8 + (lane >> 5) * 4;
    const LDS_AS char *b = (const LDS_AS char *)lds;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = *(const LDS_AS float *)(b + (k + e) * Elem<0>::MC_PITCH + m * 4);
    return v;
  }
};

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// fp32: the 16-byte fragment holds 4 k values per lane; k-slot l/32 of MFMA e uses
// element e, so four 32x32x2 MFMAs cover the same 8 k as one bf16 fragment pair.
__device__ __forceinline__ f32x16 mma(f32x4 a, f32x4 b, f32x16 c) {
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[0], b[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[1], b[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[2], b[2], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[3], b[3], c, 0, 0, 0);
  return c;
}

template <int DT, int AK, int BKIND, class Epi>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
void gemm_kernel(Operand A, Operand B, GemmGrid G, Epi epi) {
  constexpr int A_BYTES = OpLds<DT, AK>::BYTES, B_BYTES = OpLds<DT, BKIND>::BYTES;
  constexpr int STAGE = A_BYTES + B_BYTES;
  constexpr int BK = Elem<DT>::BK;
  __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];

  const int T = gridDim.x;
  const int lin = xcd_remap(blockIdx.x, T);
  const int per_split = G.ntm * G.ntn;
  const int split = lin / per_split;
  const int rem = lin - split * per_split;
  int tm, tn;
  if (G.order == 0) {
    tm = rem / G.ntn;
    tn = rem - tm * G.ntn;
  } else {
    tn = rem / G.ntm;
    tm = rem - tn * G.ntm;
  }
  const int m0 = tm * kTile, n0 = tn * kTile;
  const int kb = split * G.k_len;
  const int ke = min(G.k_total, kb + G.k_len);
  const int nk = ke > kb ? (ke - kb + BK - 1) / BK : 0;

  const int t = threadIdx.x, lane = t & 63, w = t >> 6, wr = w >> 1, wc = w & 1;

  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};

  u32x4 ra[8], rbuf[8];
  if (nk > 0) {
    load_stage<DT, AK>(ra, A, m0, kb, t);
    load_stage<DT, BKIND>(rbuf, B, n0, kb, t);
    store_stage<DT, AK>(smem, ra, t);
    store_stage<DT, BKIND>(smem + A_BYTES, rbuf, t);
  }
  __syncthreads();

  for (int it = 0; it < nk; ++it) {
    const int cur = it & 1;
    const bool more = it + 1 < nk;
    if (more) {
      load_stage<DT, AK>(ra, A, m0, kb + (it + 1) * BK, t);
      load_stage<DT, BKIND>(rbuf, B, n0, kb + (it + 1) * BK, t);
    }
    const char *la = smem + cur * STAGE;
    const char *lb = la + A_BYTES;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      typename Frag<DT, AK>::type fa[4];
      typename Frag<DT, BKIND>::type fb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) fa[i] = Frag<DT, AK>::load(la, wr * 128 + i * 32, ks, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) fb[j] = Frag<DT, BKIND>::load(lb, wc * 128 + j * 32, ks, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mma(fa[i], fb[j], acc[i][j]);
    }
    if (more) {
      char *nxt = smem + (cur ^ 1) * STAGE;
      store_stage<DT, AK>(nxt, ra, t);
      store_stage<DT, BKIND>(nxt + A_BYTES, rbuf, t);
    }
    __syncthreads();
  }
  epi(acc, m0 + wr * 128, n0 + wc * 128, lane, split, smem);
}

// Accumulator number s = (rb * NCB + cb) * 16 + i of a lane.  s is wave-uniform, so the
// switch becomes a tree of scalar branches that ends in one register move.
template <int NRB, int NCB, int S>
__device__ __forceinline__ float acc_at(const f32x16 (&acc)[NRB][NCB]) {
  if constexpr (S < NRB * NCB * 16) return acc[S / (16 * NCB)][(S / 16) % NCB][S % 16];
  else return 0.f;
}
template <int NRB, int NCB>
__device__ __forceinline__ float pick_acc(const f32x16 (&acc)[NRB][NCB], int s) {
  static_assert(NRB * NCB * 16 <= 256, "at most 256 accumulators per lane");
  switch (s) {
#define KD_ACC1(n) case n: return acc_at<NRB, NCB, n>(acc);
#define KD_ACC4(n) KD_ACC1(n) KD_ACC1(n + 1) KD_ACC1(n + 2) KD_ACC1(n + 3)
#define KD_ACC16(n) KD_ACC4(n) KD_ACC4(n + 4) KD_ACC4(n + 8) KD_ACC4(n + 12)
#define KD_ACC64(n) KD_ACC16(n) KD_ACC16(n + 16) KD_ACC16(n + 32) KD_ACC16(n + 48)
    KD_ACC64(0) KD_ACC64(64) KD_ACC64(128) KD_ACC64(192)
#undef KD_ACC64
#undef KD_ACC16
#undef KD_ACC4
#undef KD_ACC1
    default: return 0.f;
  }
}

// ---------------------------------------------------------------------------------
// bf16 MFMA GEMM core, pipelined
//
// Same tile, wave layout, operand kinds and epilogues as gemm_kernel, with:
//  * operands copied global -> LDS by the buffer unit (buffer_load_dwordx4 ... lds),
//    so no staging registers; lanes whose element lies outside the operand get an
//    offset past the buffer's range and read zero;
//  * a ring of NST LDS stages of BK k, every slot loading: the slot of the stage just
//    consumed is refilled at once, NST stages ahead;
//  * one barrier per stage, placed before the last 16-k substep, so that the fragment
//    reads for the next substep always overlap 16 MFMAs in flight.
// KC stage tile: [256 rows][2*BK B], 16-B chunk kc of row r at kc ^ swz(r).
// MC stage tile: [BK k][512 B], 16-B chunk mc of row k at chunk mc ^ ((k&3)<<2).
// The LDS serves 256 B per clock (64 banks of 4 B): a ds_read_b128 in four phases of
// 16 lanes, a ds_read_b64_tr_b16 in two phases of 32 lanes.  With these swizzles
// every phase of a fragment read touches 16 distinct 16-B bank groups.
// ---------------------------------------------------------------------------------
namespace pipe {
constexpr int OOB = (int)0x80000000;   // offset outside every buffer: reads zero
constexpr int kLoadSc1 = 16;           // buffer-load cache-policy bit SC1

// Stage geometry for a k-depth of BK bf16 (32 or 64) and ROWS tile rows (256 or 384).
template <int BK, int ROWS = 256> struct Geo {
  static constexpr int OPB = ROWS * BK * 2;  // bytes per operand per stage
  static constexpr int ROWB = BK * 2;        // KC row bytes
  static constexpr int CPR = BK / 8;         // KC 16-B chunks per row
  static constexpr int LOADS = OPB / 1024;   // 1-KB buffer loads per operand per stage
  // KC swizzle: a 16-lane LDS phase reads 16 rows of one logical chunk; rows that share
  // a 256-B bank window (same row % (256/ROWB)) get distinct chunks.
  static __device__ __forceinline__ int kc_swz(int row) {
    return BK == 32 ? ((row >> 2) & 3) : ((row >> 1) & 7);
  }
};

// Per-lane description of the NI chunks (of 16 B) one lane moves per operand per stage.
// Chunk j of wave w sits at LDS position q = (w*NI + j)*64 + lane (16-B units).
//   KC: row q / CPR, 16-B column (q % CPR) ^ swz(row);
//   MC: k row q / 32, 16-B column (q % 32) ^ ((k & 3) << 2).
// With BK = 64 (CPR = 8) and NI even, both reduce to a part shared by all chunks of one
// parity of j plus a wave-uniform part linear in g = w*NI + j, so a lane keeps two
// offsets and two k (or mn) values instead of three numbers per chunk.
template <int KIND, int BK, int NI> struct LaneChunks {
  static_assert(BK == 64 && NI % 2 == 0, "chunk parity layout");
  int rel[2];   // per-lane byte offset (even, odd j)
  int var[2];   // KC: k offset; MC: mn offset (even, odd j)
  int fix;      // KC: row within a group of 8; MC: k within a pair
  long long ld;
  __device__ __forceinline__ void init(long long ld_, int lane) {
    ld = ld_;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (KIND == OP_KC) {
        // row = 8 g + (lane >> 3); swz(row) = (row >> 1) & 7 = (4 (g & 1) + (lane >> 4)) & 7
        const int kc = (lane & 7) ^ ((4 * p + (lane >> 4)) & 7);
        fix = lane >> 3;
        var[p] = kc * 8;
        rel[p] = (int)(((long long)fix * ld + kc * 8) * 2);
      } else {
        // k = 2 g + (lane >> 5); (k & 3) = 2 (g & 1) + (lane >> 5)
        const int mc = (lane & 31) ^ ((2 * p + (lane >> 5)) << 2);
        fix = lane >> 5;
        var[p] = mc * 8;
        rel[p] = (int)(((long long)fix * ld + mc * 8) * 2);
      }
    }
  }
  // chunk g = w*NI + j of the stage: mn, k offsets within the tile / stage and the
  // byte offset from the stage base
  __device__ __forceinline__ void at(int g, int &mn, int &k, int &off) const {
    const int p = g & 1;
    if (KIND == OP_KC) {
      mn = 8 * g + fix;
      k = var[p];
      off = (int)(16LL * g * ld) + rel[p];
    } else {
      mn = var[p];
      k = 2 * g + fix;
      off = (int)(4LL * g * ld) + rel[p];
    }
  }
};

// Cache policy sc1 (device scope) on every operand load: the lines go through L2 only;
// each CU reads a line once per stage, so the vector L1 holds nothing it would reuse.
template <int KIND, int BK, int NI> struct Loader {
static __device__ __forceinline__ void issue(const Operand &op, const LaneChunks<KIND, BK, NI> &c,
                                             int mn0, int k0, char *lds, int w) {
  const unsigned short *base = (const unsigned short *)op.ptr;
  base += op_index(op, KIND, mn0, k0);   // a stage never crosses a 256-column block
  if (KIND == OP_KC && k0 + BK <= op.k_ext) {
    // The whole stage lies inside k.  The resource ends at row mn_ext, so the hardware
    // drops rows past the operand; chunk g = w*NI + j (rows 8g .. 8g+7 of the tile) is at
    // rel[g & 1] + 16 g ld bytes.  The two lane offsets are made opaque here so that the
    // per-chunk offsets are formed at each stage instead of being held in registers.
    const long long rows = (long long)op.mn_ext - mn0;
    const long long bytes = rows * op.ld * 2;
    const int nrec = rows <= 0 ? 0 : bytes > 0x7FFFFFFFLL ? 0x7FFFFFFF : (int)bytes;
    __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, nrec, 0x00020000);
    int r0 = c.rel[0], r1 = c.rel[1];
    asm volatile("" : "+v"(r0), "+v"(r1));
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int g = w * NI + j;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (LDS_AS void *)((LDS_AS char *)lds + g * 1024), 16,
          ((j & 1) ? r1 : r0) + (int)(16LL * g * op.ld), 0, 0, kLoadSc1);
    }
    return;
  }
  // general case (the last, partial stage of k, or an MC operand): per-lane tests
  __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, 0x7FFFFFFF, 0x00020000);
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    int mn, k, off;
    c.at(w * NI + j, mn, k, off);
    const bool ok = (mn0 + mn < op.mn_ext) && (k0 + k < op.k_ext);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs, (LDS_AS void *)((LDS_AS char *)lds + (w * NI + j) * 1024), 16, ok ? off : OOB, 0, 0,
        kLoadSc1);
  }
}
};

template <int KIND, int BK> struct PFrag;
template <int BK> struct PFrag<OP_KC, BK> {
  static __device__ __forceinline__ bf16x8 load(const char *lds, int r0, int ks, int lane) {
    using GG = Geo<BK>;
    const int row = r0 + (lane & 31), kc = ks * 2 + (lane >> 5);
    return *(const LDS_AS bf16x8 *)((const LDS_AS char *)lds + row * GG::ROWB +
                                    ((kc ^ GG::kc_swz(row)) << 4));
  }
};
template <int BK> struct PFrag<OP_MC, BK> {
  static __device__ __forceinline__ bf16x8 load(const char *lds, int r0, int ks, int lane) {
    const int s = lane & 15, g = lane >> 4;
    const int m = r0 + (g & 1) * 16 + 4 * (s & 3);
    const int k = ks * 16 + (g >> 1) * 8 + (s >> 2);
    const int col = (((m >> 3) ^ ((k & 3) << 2)) << 4) + (m & 7) * 2;
    const LDS_AS char *b = (const LDS_AS char *)lds;
    s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s16x4 *)(b + k * 512 + col));
    s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s16x4 *)(b + (k + 4) * 512 + col));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// s_waitcnt with vmcnt <= N and, with LGKM0, lgkmcnt == 0.  Immediate: vmcnt in bits
// 3:0 and 15:14, expcnt 6:4 and lgkmcnt 11:8 (left at their maxima unless LGKM0).
template <int N, bool LGKM0>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt is six bits");
  __builtin_amdgcn_s_waitcnt((LGKM0 ? 0x0070 : 0x0F70) | (N & 15) | ((N >> 4) << 14));
}
}  // namespace pipe

// Scheduling hints: sched_group_barrier(mask, n, id) asks the scheduler for the next
// n instructions of a class; the sequence below places one load or LDS read in the
// shadow of each MFMA, so that with one wave per SIMD the matrix core never waits for
// the wave to issue its memory traffic.
#define KD_SG_MFMA 0x008
#define KD_SG_VALU 0x002
#define KD_SG_SALU 0x004
#define KD_SG_VMEM 0x020
#define KD_SG_DSRD 0x100

// WN = waves along n: 2 gives 4 waves of (TMA/2) x 128 (one per SIMD), 4 gives 8 waves
// of (TMA/2) x 64 (two per SIMD, so one wave's MFMAs cover the other's waits).  TMA =
// rows of the A tile: 256, or 384 for a k-contiguous A, which cuts the operand bytes
// per flop by a sixth; with TMA = 384 the A fragments are single-buffered (each one is
// re-read for the next substep as soon as its MFMAs have issued) so that the 192
// accumulators per lane and the fragments fit in 256 registers.  NSTA / NSTB = LDS
// slots of the A / B rings; A may have one slot more than B.
template <int AK, int BKIND, class Epi, int NSTA, int NSTB, int BK, int WN, int TMA = 256>
__global__ __attribute__((amdgpu_flat_work_group_size(128 * WN, 128 * WN),
                          amdgpu_waves_per_eu(WN / 2, WN / 2)))
void gemm_pipe_kernel(Operand A, Operand B, GemmGrid G, Epi epi) {
  using namespace pipe;
  using GA = Geo<BK, TMA>;
  using GB = Geo<BK, 256>;
  constexpr int NW = 2 * WN;            // waves
  constexpr int NCB = 8 / WN;           // 32-column MFMA blocks per wave
  constexpr int WNC = 32 * NCB;         // columns per wave
  constexpr int WMR = TMA / 2;          // rows per wave
  constexpr int NRB = WMR / 32;         // 32-row MFMA blocks per wave
  constexpr int NIA = GA::LOADS / NW;   // buffer loads per wave per stage, A
  constexpr int NIB = GB::LOADS / NW;   // buffer loads per wave per stage, B
  constexpr int S = BK / 16;            // 16-k substeps per stage
  constexpr int LPS = NIA + NIB;        // buffer loads per wave per stage
  constexpr int NMF = NRB * NCB;        // MFMAs per wave per substep
  constexpr bool FA1 = TMA > 256;       // single-buffered A fragments
  // LDS reads per substep: one per fragment, two per transposed (MC) fragment
  constexpr int NRD = NRB * (AK == OP_MC ? 2 : 1) + NCB * (BKIND == OP_MC ? 2 : 1);
  static_assert(NSTB >= 2 && (NSTA == NSTB || NSTA == NSTB + 1), "ring shapes");
  static_assert(TMA == 256 || (TMA == 384 && AK == OP_KC), "a 384-row A tile must be k-contiguous");
  static_assert(GA::LOADS % NW == 0 && GB::LOADS % NW == 0, "whole loads per wave");
  __shared__ __attribute__((aligned(1024))) char smem[NSTA * GA::OPB + NSTB * GB::OPB];
  char *const smemB = smem + NSTA * GA::OPB;

  const int lin = xcd_remap(blockIdx.x, gridDim.x);
  const int per_split = G.ntm * G.ntn;
  const int split = lin / per_split;
  const int rem = lin - split * per_split;
  int tm, tn;
  if (G.order == 0) {
    if (G.ngrp > 0 && G.ngrp < G.ntn) {
      const int span = G.ntm * G.ngrp, grp = rem / span;
      const int gs = min(G.ngrp, G.ntn - grp * G.ngrp), r = rem - grp * span;
      tm = r / gs;
      tn = grp * G.ngrp + (r - tm * gs);
    } else {
      tm = rem / G.ntn;
      tn = rem - tm * G.ntn;
    }
  } else {
    tn = rem / G.ntm;
    tm = rem - tn * G.ntm;
  }
  const int m0 = tm * TMA, n0 = tn * kTile;
  const int kb = split * G.k_len;
  const int ke = min(G.k_total, kb + G.k_len);
  const int nk = ke > kb ? (ke - kb + BK - 1) / BK : 0;

  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wr = w / WN, wc = w % WN;
  LaneChunks<AK, BK, NIA> ca;
  LaneChunks<BKIND, BK, NIB> cb;
  ca.init(A.ld, lane);
  cb.init(B.ld, lane);
  // k beyond this split's range reads zero (and moves no data)
  Operand Ak = A, Bk = B;
  Ak.k_ext = min(A.k_ext, ke);
  Bk.k_ext = min(B.k_ext, ke);

  f32x16 acc[NRB][NCB];
#pragma unroll
  for (int i = 0; i < NRB; ++i)
#pragma unroll
    for (int j = 0; j < NCB; ++j) acc[i][j] = f32x16{};

  // Prologue: every slot loading, in the order A0 B0 A1 B1 [A2] (stages past the end
  // are all-zero loads, so the count of loads in flight is the same in every
  // iteration); then stage 0 landed.
  for (int s = 0; s < NSTA; ++s) {
    Loader<AK, BK, NIA>::issue(Ak, ca, m0, kb + s * BK, smem + s * GA::OPB, w);
    if (s < NSTB) Loader<BKIND, BK, NIB>::issue(Bk, cb, n0, kb + s * BK, smemB + s * GB::OPB, w);
  }
  // epilogue inputs that do not depend on the product, loaded behind the first stages
  typename Epi::Pre pre{};
  if constexpr (Epi::kPrefetch) pre = epi.template prefetch<NRB>(m0 + wr * WMR, n0 + wc * WNC);
  wait_vm<NIA * (NSTA - 1) + NIB * (NSTB - 1), false>();
  __syncthreads();

  constexpr int NFA = FA1 ? 1 : 2;
  bf16x8 fa[NFA][NRB], fb[2][NCB];
#pragma unroll
  for (int i = 0; i < NRB; ++i) fa[0][i] = PFrag<AK, BK>::load(smem, wr * WMR + i * 32, 0, lane);
#pragma unroll
  for (int j = 0; j < NCB; ++j) fb[0][j] = PFrag<BKIND, BK>::load(smemB, wc * WNC + j * 32, 0, lane);

  int acur = 0, bcur = 0;  // ring slots of stage it
  for (int it = 0; it < nk; ++it) {
    const int anext = acur + 1 == NSTA ? 0 : acur + 1;
    const int bnext = bcur + 1 == NSTB ? 0 : bcur + 1;
    char *cura = smem + acur * GA::OPB;
    char *curb = smemB + bcur * GB::OPB;
#pragma unroll
    for (int ss = 0; ss < S - 1; ++ss) {
      // substep ss on registers [ss&1]; read substep ss+1 meanwhile
#pragma unroll
      for (int j = 0; j < NCB; ++j)
        fb[(ss + 1) & 1][j] = PFrag<BKIND, BK>::load(curb, wc * WNC + j * 32, ss + 1, lane);
      if constexpr (FA1) {
#pragma unroll
        for (int i = 0; i < NRB; ++i) {
#pragma unroll
          for (int j = 0; j < NCB; ++j) acc[i][j] = mma(fa[0][i], fb[ss & 1][j], acc[i][j]);
          fa[0][i] = PFrag<AK, BK>::load(cura, wr * WMR + i * 32, ss + 1, lane);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NRB; ++i)
          fa[(ss + 1) & 1][i] = PFrag<AK, BK>::load(cura, wr * WMR + i * 32, ss + 1, lane);
#pragma unroll
        for (int i = 0; i < NRB; ++i)
#pragma unroll
          for (int j = 0; j < NCB; ++j) acc[i][j] = mma(fa[ss & 1][i], fb[ss & 1][j], acc[i][j]);
      }
      // one or two LDS reads in the shadow of each MFMA
#pragma unroll
      for (int q = 0; q < NMF; ++q) {
        __builtin_amdgcn_sched_group_barrier(KD_SG_MFMA, 1, 0);
        __builtin_amdgcn_sched_group_barrier(KD_SG_DSRD, (NRD + NMF - 1) / NMF, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }

    // Stage it+1 must have landed for every wave, and every wave must hold the whole of
    // stage it in registers or accumulators, since its slots are refilled next.  Loads
    // are issued B(j+NSTB) then A(j+NSTA) in iteration j, so what may still be in
    // flight here is A(it+2) when A has the extra slot, else nothing.
    wait_vm<NIA * (NSTA - NSTB), true>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);

    // last substep on registers [(S-1)&1]; meanwhile read substep 0 of stage it+1 and
    // refill this stage's slots with B(it+NSTB) and A(it+NSTA)
    const char *nxa = smem + anext * GA::OPB;
    const char *nxb = smemB + bnext * GB::OPB;
#pragma unroll
    for (int j = 0; j < NCB; ++j) fb[0][j] = PFrag<BKIND, BK>::load(nxb, wc * WNC + j * 32, 0, lane);
    if constexpr (FA1) {
#pragma unroll
      for (int i = 0; i < NRB; ++i) {
#pragma unroll
        for (int j = 0; j < NCB; ++j) acc[i][j] = mma(fa[0][i], fb[(S - 1) & 1][j], acc[i][j]);
        fa[0][i] = PFrag<AK, BK>::load(nxa, wr * WMR + i * 32, 0, lane);
      }
      Loader<BKIND, BK, NIB>::issue(Bk, cb, n0, kb + (it + NSTB) * BK, curb, w);
      Loader<AK, BK, NIA>::issue(Ak, ca, m0, kb + (it + NSTA) * BK, cura, w);
    } else {
#pragma unroll
      for (int i = 0; i < NRB; ++i) fa[0][i] = PFrag<AK, BK>::load(nxa, wr * WMR + i * 32, 0, lane);
      Loader<BKIND, BK, NIB>::issue(Bk, cb, n0, kb + (it + NSTB) * BK, curb, w);
      Loader<AK, BK, NIA>::issue(Ak, ca, m0, kb + (it + NSTA) * BK, cura, w);
#pragma unroll
      for (int i = 0; i < NRB; ++i)
#pragma unroll
        for (int j = 0; j < NCB; ++j)
          acc[i][j] = mma(fa[(S - 1) & 1][i], fb[(S - 1) & 1][j], acc[i][j]);
    }
    // reads for the next stage in the first half of the MFMAs (they gate the next
    // iteration), loads in the second half
#pragma unroll
    for (int q = 0; q < NMF / 2; ++q) {
      __builtin_amdgcn_sched_group_barrier(KD_SG_MFMA, 1, 1);
      __builtin_amdgcn_sched_group_barrier(KD_SG_DSRD, (2 * NRD + NMF - 1) / NMF, 1);
    }
#pragma unroll
    for (int q = 0; q < NMF / 2; ++q) {
      __builtin_amdgcn_sched_group_barrier(KD_SG_MFMA, 1, 1);
      __builtin_amdgcn_sched_group_barrier(KD_SG_VMEM, (2 * LPS + NMF - 1) / NMF, 1);
      __builtin_amdgcn_sched_group_barrier(KD_SG_VALU, 2, 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    acur = anext;
    bcur = bnext;
  }
  wait_vm<0, false>();  // the zero loads issued past the end
  if constexpr (Epi::kPrefetch)
    epi(acc, m0 + wr * WMR, n0 + wc * WNC, lane, split, smem, pre);
  else
    epi(acc, m0 + wr * WMR, n0 + wc * WNC, lane, split, smem);
}

template <int DT, int AK, int BKIND, class Epi>
static hipError_t run_gemm(const Operand &A, const Operand &B, const GemmGrid &G, const Epi &epi,
                           hipStream_t s) {
  const long long T = (long long)G.ntm * G.ntn * G.nsplit;
  if (T <= 0) return hipSuccess;
  // 8 waves (two per SIMD), two LDS stages of 64 k: a KC operand row is then one
  // 128-byte segment per stage, which halves the memory requests of k-contiguous operands
  if constexpr (DT == 1)
    hipLaunchKernelGGL((gemm_pipe_kernel<AK, BKIND, Epi, 2, 2, 64, 4, kTileA16>), dim3((unsigned)T),
                       dim3(512), 0, s, A, B, G, epi);
  else
    hipLaunchKernelGGL((gemm_kernel<DT, AK, BKIND, Epi>), dim3((unsigned)T), dim3(256), 0, s, A,
                       B, G, epi);
  return hipGetLastError();
}

static inline int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

}  // namespace kd
