// Log probabilities of given tokens from rows of logits, with the entropy, the logsumexp
// and the largest alternatives, and their gradient.
//
// For a row z with m = max z, S = sum exp(z - m), T = sum exp(z - m) (z - m):
//   lse = m + ln S,  ln p_v = z_v - m - ln S,  H = -sum p ln p = ln S - T / S.
// One pass: every lane keeps its own (m, S, T) and rescales the sums when its maximum
// rises; lanes, waves and vocabulary splits are joined by the same rule in double.
//
// Bound by reading the logits once: 4096 rows of 128256 bf16 logits (1.05 GB) take 181 us, 5.8
// TB/s, and 197 us with 8 alternatives; 1037 rows of 32003 float32 logits, a third of them
// masked, 26 us (5.1 TB/s).  Few rows are bound by latency: one row of 128256 takes 5.3 us in
// two launches (the splits and their join), 13.1 us with 20 alternatives, whose selection is a
// chain of short dependent steps in each.
#include "kd_ops.h"

#include <cstdint>
#include <cstring>
#include <type_traits>

namespace kd {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpSlots = 4;  // 16-byte loads in flight per thread and step

template <int DT> struct LpT;
template <> struct LpT<1> { static constexpr int EPL = 8, ES = 2; };
template <> struct LpT<0> { static constexpr int EPL = 4, ES = 4; };

typedef unsigned int u4 __attribute__((ext_vector_type(4)));
#define LDS_AS __attribute__((address_space(3)))

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

// The value of lane ^ J, J a power of two: data-parallel moves inside 16 lanes, row and half
// swaps beyond, so that a sorting stage waits a few cycles instead of an LDS round trip.
template <int J>
__device__ __forceinline__ unsigned lane_xor(unsigned v, int lane) {
  if constexpr (J == 1) return __builtin_amdgcn_update_dpp(0u, v, 0xB1, 0xF, 0xF, true);
  else if constexpr (J == 2) return __builtin_amdgcn_update_dpp(0u, v, 0x4E, 0xF, 0xF, true);
  else if constexpr (J == 4) {  // reversed in eights, then in fours
    const unsigned r = __builtin_amdgcn_update_dpp(0u, v, 0x141, 0xF, 0xF, true);
    return __builtin_amdgcn_update_dpp(0u, r, 0x1B, 0xF, 0xF, true);
  } else if constexpr (J == 8) return __builtin_amdgcn_update_dpp(0u, v, 0x128, 0xF, 0xF, true);
  else if constexpr (J == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (lane & 16) ? r[0] : r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (lane & 32) ? r[0] : r[1];
  }
}
template <int J>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v, int lane) {
  return ((uint64_t)lane_xor<J>((unsigned)(v >> 32), lane) << 32) | lane_xor<J>((unsigned)v, lane);
}
// One stage: lanes with keep_max keep the larger of the pair.
template <int J, class K>
__device__ __forceinline__ K sort_stage(K v, int lane, bool keep_max) {
  const K o = lane_xor<J>(v, lane);
  return (v > o) == keep_max ? v : o;
}
template <int J, class K>
__device__ __forceinline__ K sort_down(K v, int lane, bool desc) {
  v = sort_stage<J>(v, lane, ((lane & J) == 0) == desc);
  if constexpr (J > 1) v = sort_down<J / 2>(v, lane, desc);
  return v;
}
// Bitonic sort of the wave's 64 keys, descending over the lanes.
template <class K>
__device__ __forceinline__ K wave_sort(K v, int lane) {
  v = sort_down<1>(v, lane, (lane & 2) == 0);
  v = sort_down<2>(v, lane, (lane & 4) == 0);
  v = sort_down<4>(v, lane, (lane & 8) == 0);
  v = sort_down<8>(v, lane, (lane & 16) == 0);
  v = sort_down<16>(v, lane, (lane & 32) == 0);
  return sort_down<32>(v, lane, true);
}
// A value that at least n <= 64 of the wave's 64 U maxima reach: their n-th largest, found bit by
// bit from the top by counting and cut off after 16 bits (all there are in bf16).
template <int U>
__device__ __forceinline__ float wave_nth(const float (&x)[U], int n) {
  unsigned key[U], t = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) key[u] = val_key(x[u]);
#pragma unroll 1
  for (unsigned bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
    int c = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) c += __popcll(__builtin_amdgcn_ballot_w64(key[u] >= (t | bit)));
    if (c >= n) t |= bit;
    if (c == n) break;
  }
  return t > val_key(-INFINITY) ? key_val(t) : -INFINITY;
}
__device__ __forceinline__ uint64_t shfl64(uint64_t v, int l) {
  const unsigned lo = __shfl((unsigned)v, l, 64), hi = __shfl((unsigned)(v >> 32), l, 64);
  return ((uint64_t)hi << 32) | lo;
}
// The 64 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t wave_merge(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = shfl64(b, 63 - lane);
  return sort_down<32>(a > r ? a : r, lane, true);  // the larger ones are bitonic
}
// Of n keys in LDS, any order, the 64 largest, descending.
__device__ __forceinline__ uint64_t wave_best(const LDS_AS uint64_t *keys, int n, int lane) {
  uint64_t list = 0;
  for (int i = 0; i < n; i += 64) {
    const uint64_t v = wave_sort(i + lane < n ? keys[i + lane] : (uint64_t)0, lane);
    list = i == 0 ? v : wave_merge(list, v, lane);
  }
  return list;
}

// A wave's candidates for the row's `top` largest.  The streaming loop only notes, in LDS,
// which groups of elements hold one (a compare of the group's maximum and a few instructions
// where it passes); the groups are read again when a wave's worth of them has come together,
// which is a few dozen of a row's thousands.
// An element is a candidate if it is above the threshold, or equal to it with an index below
// `tie`.  Every threshold is a value that at least `top` elements of the row reach: the top-th
// largest of the running maxima of 64 lanes x 4 slots, another wave's threshold (ties are let
// in), or, where the buffer was cut back to its largest, the top-th of those (ties with a larger
// index are not).
// Up to kLpFew alternatives take the threshold from the 64 lanes' maxima, one sort of them
// (200000 float32 logits, 5: 11 us against 15); more from the maxima of lanes and slots, which
// are not as close to the top-th largest of a lane (60000 logits, 50: 20 us against 23).
constexpr int kLpFew = 24;
constexpr int kLpBuf = 256;   // keys of candidates per wave
constexpr int kLpNotes = 384; // noted groups per wave: room for a whole step is kept
struct WaveTop {
  float thr;
  unsigned tie;
  int cnt, notes, masked, top, lane;
  // the wave's own: fences stand between its lanes' writes and reads (volatile accesses would
  // each be waited for)
  LDS_AS uint64_t *buf;
  LDS_AS unsigned *note;
  __device__ __forceinline__ void init(int top_, int epl, int lane_, LDS_AS uint64_t *b,
                                       LDS_AS unsigned *n) {
    thr = -INFINITY;
    masked = (top_ + epl - 1) / epl;
    tie = ~0u;
    cnt = notes = 0;
    top = top_;
    lane = lane_;
    buf = b;
    note = n;
  }
  __device__ __forceinline__ void raise(float v) {
    if (v > thr) {
      thr = v;
      tie = ~0u;
    }
  }
  __device__ __forceinline__ void cut() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const uint64_t list = wave_best(buf, cnt, lane);
    cnt = __popcll(__builtin_amdgcn_ballot_w64(list != 0 && lane < top));
    if (lane < cnt) buf[lane] = list;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const unsigned hi = __builtin_amdgcn_readlane((unsigned)(list >> 32), top - 1);
    const unsigned lo = __builtin_amdgcn_readlane((unsigned)list, top - 1);
    if (hi != 0 && key_val(hi) >= thr) {
      thr = key_val(hi);
      tie = ~lo;
    }
  }
  __device__ __forceinline__ bool above(float x, unsigned idx) const {
    return x > thr || (x == thr && idx < tie);
  }
  // Lanes below this one in the mask.
  static __device__ __forceinline__ int prefix(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((unsigned)(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo((unsigned)mask, 0));
  }
  // Notes the group at index idx whose maximum is mx, if it can hold a candidate.
  __device__ __forceinline__ void look(float mx, unsigned idx) {
    bool in = above(mx, idx);
    uint64_t mask = __builtin_amdgcn_ballot_w64(in);
    if (mask == 0) return;
    // masked groups (all -inf, in index order): the first `top` elements' worth is enough
    const uint64_t none = __builtin_amdgcn_ballot_w64(in && mx == -INFINITY);
    if (none) {
      in = in && (mx > -INFINITY || prefix(none) < masked);
      masked -= min(masked, (int)__popcll(none));
      mask = __builtin_amdgcn_ballot_w64(in);
    }
    if (in) note[notes + prefix(mask)] = idx;
    notes += __popcll(mask);
  }
  // Reads the noted groups (at: from index to address; end: the range's) and keeps their
  // candidates, `most` of them at the end.
  template <int DT, class At>
  __device__ __forceinline__ void drain(unsigned end, int most, At at) {
    constexpr int EPL = LpT<DT>::EPL;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    bool has = false;
    unsigned e = 0, from = 0;
    u4 r = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int i = 0, j = EPL;; ++j) {
      const bool done = j == EPL && i >= notes;
      if (j == EPL && !done) {  // the next groups, one per lane
        has = i + lane < notes;
        e = has ? note[i + lane] : 0u;
        // a group at the end is read from the last whole group's place: skip what precedes it
        from = has && e + EPL <= end ? e : end - EPL;
        r = load16(at(from));
        i += 64;
        j = 0;
        float x[EPL];
        unpack<DT>(r, x);
        uint64_t in[EPL];
        int all = cnt;
#pragma unroll
        for (int q = 0; q < EPL; ++q) {
          in[q] = __builtin_amdgcn_ballot_w64(has && from + q >= e && above(x[q], from + q));
          all += __popcll(in[q]);
        }
        if (all <= kLpBuf) {  // nearly always: no cut between them
#pragma unroll
          for (int q = 0; q < EPL; ++q) {
            if (in[q] >> lane & 1) buf[cnt + prefix(in[q])] = sel_key(x[q], from + q);
            cnt += __popcll(in[q]);
          }
          j = EPL - 1;
          continue;
        }
      }
      // room for 64 more (the cut is long, and so in one place)
      if (cnt > (done ? most : kLpBuf - 64)) cut();
      if (done) break;
      const float x = __uint_as_float(DT == 0 ? r[0] : r[0] << 16);
      const bool in = has && from + j >= e && above(x, from + j);
      const uint64_t mask = __builtin_amdgcn_ballot_w64(in);
      if (in) buf[cnt + prefix(mask)] = sel_key(x, from + j);
      cnt += __popcll(mask);
      if (DT == 0) {
        r = u4{r[1], r[2], r[3], 0u};
      } else {
        r = u4{(r[0] >> 16) | (r[1] << 16), (r[1] >> 16) | (r[2] << 16),
               (r[2] >> 16) | (r[3] << 16), r[3] >> 16};
      }
    }
    notes = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
};

// Partial sums of one vocabulary split of a row.
struct LpPart {
  double S, T;
  float m;
  int pad;
};

constexpr float kLpNone = -3.4028234663852886e38f;  // m before the first value

// Joins (m2, S2, T2) to (m, S, T).
__device__ __forceinline__ void lp_join(float &m, double &S, double &T, float m2, double S2,
                                        double T2) {
  const float M = __builtin_elementwise_maximum(m, m2);  // NaN stays
  const float d1 = fmaxf(m - M, kOpLowest), d2 = fmaxf(m2 - M, kOpLowest);
  const double c1 = (double)__builtin_amdgcn_exp2f(d1 * kOpLog2e);
  const double c2 = (double)__builtin_amdgcn_exp2f(d2 * kOpLog2e);
  T = c1 * (T + (double)d1 * S) + c2 * (T2 + (double)d2 * S2);
  S = c1 * S + c2 * S2;
  m = M;
}
__device__ __forceinline__ void wave_join(float &m, double &S, double &T) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float m2 = __shfl_xor(m, o, 64);
    const double S2 = __shfl_xor(S, o, 64), T2 = __shfl_xor(T, o, 64);
    lp_join(m, S, T, m2, S2, T2);
  }
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

// The row's r-th alternative (key 0: there is none, in a bad row).
__device__ __forceinline__ void write_top(const LpOut &o, long long row, int top, int r,
                                          uint64_t key, float m, float lnS) {
  const float nan = __uint_as_float(0x7FC00000u);
  const bool bad = lnS != lnS, empty = lnS == -INFINITY;
  const float x = key_val((unsigned)(key >> 32));
  o.top_idx[row * top + r] = bad ? -1 : (int32_t)~(unsigned)key;
  o.top_logp[row * top + r] = bad ? nan : empty ? -INFINITY : (x - m) - lnS;
}

// Hands the `top` largest of n unique keys in LDS (any order) to f(rank, key), a key per thread
// and its rank by counting the larger ones; ranks from n on get key 0.  All NT threads.
template <int NT, class F>
__device__ __forceinline__ void place_top(const uint64_t *keys, int n, int top, int t, F f) {
  for (int i = t; i < n; i += NT) {
    const uint64_t key = keys[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += keys[j] > key ? 1 : 0;
    if (rank < top) f(rank, key);
  }
  for (int r = n + t; r < top; r += NT) f(r, 0ull);
}

template <int DT>
__device__ __forceinline__ float logit_at(const char *row, long long v) {
  return DT == 0 ? ((const float *)row)[v]
                 : __uint_as_float((unsigned)((const unsigned short *)row)[v] << 16);
}

// One workgroup of NT threads per (row, vocabulary split).  A step is U 16-byte groups per
// thread, loaded one step ahead.  Past the end a group is loaded from the range's last 16
// bytes instead and what earlier groups hold is masked, so no load is conditional or leaves
// the range (of at least one group).
template <int DT, bool TOP, int NT, int U>
__global__ __launch_bounds__(NT) void k_token_logprobs(LpArgs a) {
  constexpr int EPL = LpT<DT>::EPL, ES = LpT<DT>::ES, NW = NT / 64;
  __shared__ float s_m[NW], s_thr[NW];
  __shared__ double s_S[NW], s_T[NW];
  __shared__ uint64_t s_buf[TOP ? NW * kLpBuf : 1], s_pool[TOP ? NW * kLpBuf : 1];
  __shared__ unsigned s_note[TOP ? NW * kLpNotes : 1];
  __shared__ int s_n;

  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const unsigned row = blockIdx.x / a.S, split = blockIdx.x - row * a.S;
  const char *rp = (const char *)a.logits + row * a.ld * ES;
  const long long e0 = split * a.per;
  const int len = (int)(e0 + a.per < a.V ? a.per : a.V - e0);  // below 2^29
  const char *sp = rp + e0 * ES;
  long long tok = -1;
  float zt = 0.f;
  if (t == 0 && a.S == 1) {
    tok = a.tokens.at(row);
    if (tok >= 0 && tok < a.V) zt = logit_at<DT>(rp, tok);
  }

  float m = kLpNone;
  double S = 0.0, T = 0.0;
  WaveTop wt;
  int fresh = 0;  // groups noted since the wave's threshold was last renewed
  float run[U];   // the largest element so far at each lane and slot
#pragma unroll
  for (int u = 0; u < U; ++u) run[u] = -INFINITY;
  if (TOP) {
    wt.init(a.top, EPL, lane, (LDS_AS uint64_t *)s_buf + w * kLpBuf,
            (LDS_AS unsigned *)s_note + w * kLpNotes);
    if (t < NW) s_thr[t] = -INFINITY;
    if (t == 0) s_n = 0;
    __syncthreads();
  }

  const unsigned last = (unsigned)(len - EPL) * ES;
  auto load = [&](u4 (&r)[U], int step) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned off = ((unsigned)(step * U + u) * NT + t) * 16u;
      r[u] = load16(sp + (off < last ? off : last));
    }
  };
  float lu[U];  // the maxima of the step's groups, NaN where a group holds nothing new
  // whole: every element of the step's groups is inside the range
  auto take = [&](const u4 (&raw)[U], int step, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    float x[U][EPL], lm = -INFINITY;  // the maximum of all, NaN if an element is
#pragma unroll
    for (int u = 0; u < U; ++u) {
      unpack<DT>(raw[u], x[u]);
      if (!WHOLE && (step * U + u) * NT * EPL >= len) {  // the same for the workgroup
        lu[u] = NAN;
        continue;
      }
      int first = 0;  // of the group's elements, those from here on are new
      if (!WHOLE) {
        const int e = ((step * U + u) * NT + t) * EPL;
        first = e <= len - EPL ? 0 : e - (len - EPL);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          if (j < first) x[u][j] = -INFINITY;
      }
      lu[u] = x[u][0];
#pragma unroll
      for (int j = 1; j < EPL; ++j) lu[u] = __builtin_elementwise_maximum(lu[u], x[u][j]);
      lm = __builtin_elementwise_maximum(lm, lu[u]);
      if (!WHOLE && first >= EPL) lu[u] = NAN;
    }
    if (!(lm <= m)) {  // also where the lane has met a NaN, which then stays
      lm = __builtin_elementwise_maximum(lm, m);
      const float d = fmaxf(m - lm, kOpLowest);
      const double c = (double)__builtin_amdgcn_exp2f(d * kOpLog2e);
      T = c * (T + (double)d * S);
      S = c * S;
      m = lm;
    }
    float ps = 0.f, pt = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!WHOLE && (step * U + u) * NT * EPL >= len) continue;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const float d = fmaxf(x[u][j] - m, kOpLowest);
        const float e = __builtin_amdgcn_exp2f(d * kOpLog2e);
        ps += e;
        pt = fmaf(e, d, pt);
      }
    }
    S += (double)ps;
    T += (double)pt;
  };
  // The step's groups among the candidates; code that is kept in one place, as it is long and
  // seldom runs.
  auto choose = [&](int step, bool end) {
#pragma unroll
    for (int u = 0; u < U; ++u) run[u] = fmaxf(run[u], lu[u]);
    if (step == 0 || fresh >= 16) {  // the maxima have grown since the last look
      if (a.top <= kLpFew) {
        float lm = run[0];
#pragma unroll
        for (int u = 1; u < U; ++u) lm = fmaxf(lm, run[u]);
        wt.raise(key_val(__builtin_amdgcn_readlane(wave_sort(val_key(lm), lane), a.top - 1)));
      } else {
        wt.raise(wave_nth(run, a.top));
      }
      if (lane == 0)
        __hip_atomic_store(&s_thr[w], wt.thr, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      fresh = 0;
    }
#pragma unroll
    for (int i = 0; i < NW; ++i)
      wt.raise(__hip_atomic_load(&s_thr[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP));
    const int before = wt.notes;
#pragma unroll
    for (int u = 0; u < U; ++u)
      wt.look(lu[u], (unsigned)e0 + ((step * U + u) * NT + t) * EPL);
    fresh += wt.notes - before;
    if (wt.notes > kLpNotes - 64 * U || end)
      wt.template drain<DT>((unsigned)e0 + len, a.S > 1 ? kLpBuf : 64,
                            [&](unsigned i) { return rp + (size_t)i * ES; });
  };

  if (len >= EPL) {
    constexpr int STEP = NT * U * EPL;
    const int whole = len / STEP, steps = (len + STEP - 1) / STEP;
    u4 cur[U], nxt[U];
    load(cur, 0);
    for (int i = 0; i < steps; ++i) {
      load(nxt, i + 1);
      if (i < whole) take(cur, i, std::true_type());
      else take(cur, i, std::false_type());
      if (TOP) choose(i, i + 1 == steps);
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = nxt[u];
    }
  } else if (w == 0) {  // fewer elements than one group: one per lane
    float x = -INFINITY;
    if (lane < len) x = logit_at<DT>(sp, lane);
    m = x > kLpNone || x != x ? x : kLpNone;
    S = x == -INFINITY ? 0.0 : 1.0;
    if (TOP) {
      if (lane < len) wt.buf[lane] = sel_key(x, (unsigned)e0 + lane);
      wt.cnt = len;
    }
  }

  wave_join(m, S, T);
  if (lane == 0) {
    s_m[w] = m;
    s_S[w] = S;
    s_T[w] = T;
    if (TOP)
      __hip_atomic_store(&s_thr[w], wt.thr, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  }
  __syncthreads();
  const long long at = (long long)row * a.S + split;
  if (TOP) {
    // the waves' candidates that reach the best threshold
    float thr = s_thr[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) thr = fmaxf(thr, s_thr[i]);
    for (int i = lane; i < wt.cnt; i += 64) {
      const uint64_t key = wt.buf[i];
      if (key_val((unsigned)(key >> 32)) >= thr) s_pool[atomicAdd(&s_n, 1)] = key;
    }
  }
  if (TOP) __syncthreads();
  if (TOP && a.S > 1)  // `top` keys, fewer only where NaN has taken the place of values
    place_top<NT>(s_pool, s_n, a.top, t, [&](int r, uint64_t key) { a.keys[at * a.top + r] = key; });
  // many rows: the other waves make room for the next ones
  if (w != 0) return;
  for (int i = 1; i < NW; ++i) lp_join(m, S, T, s_m[i], s_S[i], s_T[i]);
  if (a.S > 1) {
    if (lane == 0) a.part[at] = LpPart{S, T, m, 0};
    return;
  }
  float lnS = 0.f;
  if (lane == 0) {
    lnS = lp_log(m, S);
    lp_finish(a.out, row, m, S, T, lnS, tok, a.V, zt);
  }
  if (TOP) {
    lnS = __shfl(lnS, 0, 64);
    auto write = [&](int r, uint64_t key) { write_top(a.out, row, a.top, r, key, m, lnS); };
    const int n = s_n;
    if (n <= 64) {
      place_top<64>(s_pool, n, a.top, lane, write);
    } else {
      const uint64_t list = wave_best((const LDS_AS uint64_t *)s_pool, n, lane);
      if (lane < a.top) write(lane, list);
    }
  }
}

// Joins a row's vocabulary splits: one workgroup per row.
constexpr int kLpMaxSplits = 64;
template <int DT, bool TOP>
__global__ __launch_bounds__(kLpThreads) void k_token_logprobs_join(LpArgs a) {
  constexpr int MAXK = kLpMaxSplits * kLpMaxTop, NK = MAXK / kLpThreads;
  __shared__ uint64_t s_pool[TOP ? MAXK : 1];
  __shared__ uint64_t s_thr[kLpThreads / 64];
  __shared__ float s_row[2];
  __shared__ int s_n;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const long long row = blockIdx.x;
  const int n = TOP ? a.S * a.top : 0;
  uint64_t k[NK];
  if (TOP) {
#pragma unroll
    for (int i = 0; i < NK; ++i)
      k[i] = i * kLpThreads + t < n ? a.keys[row * n + i * kLpThreads + t] : 0ull;
  }
  float m = kLpNone, zt = 0.f;
  double S = 0.0, T = 0.0;
  long long tok = -1;
  if (w == 0) {
    if (lane < a.S) {
      const LpPart p = a.part[row * a.S + lane];
      m = p.m;
      S = p.S;
      T = p.T;
    }
    tok = a.tokens.at(row);
    if (tok >= 0 && tok < a.V)
      zt = logit_at<DT>((const char *)a.logits + row * a.ld * LpT<DT>::ES, tok);
    if (lane == 0) s_n = 0;
  }
  if (TOP) {
    // a value that `top` keys reach: of the maxima of a wave's 64 lanes x 4 sets of keys
    float best[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      unsigned b = 0;
#pragma unroll
      for (int i = u; i < NK; i += 4) b = max(b, (unsigned)(k[i] >> 32));
      best[u] = b ? key_val(b) : -INFINITY;
    }
    // (and, where many are equal, a key that `top` reach: of the maxima of its 64 lanes)
    uint64_t bound = 1, mine = 0;
    if (n > kLpThreads) {
      const float v = a.top > kLpFew ? wave_nth(best, a.top) : -INFINITY;
      bound = v > -INFINITY ? (uint64_t)val_key(v) << 32 : 1;
#pragma unroll
      for (int i = 0; i < NK; ++i) mine = k[i] > mine ? k[i] : mine;
      mine = wave_sort(mine, lane);
    }
    if (lane == a.top - 1) s_thr[w] = mine > bound ? mine : bound;
    __syncthreads();
    uint64_t thr = s_thr[0];
#pragma unroll
    for (int i = 1; i < kLpThreads / 64; ++i) thr = s_thr[i] > thr ? s_thr[i] : thr;
#pragma unroll
    for (int i = 0; i < NK; ++i)
      if (k[i] >= thr) s_pool[atomicAdd(&s_n, 1)] = k[i];
  }
  if (w == 0) {
    wave_join(m, S, T);
    if (lane == 0) {
      const float lnS = lp_log(m, S);
      lp_finish(a.out, row, m, S, T, lnS, tok, a.V, zt);
      s_row[0] = m;
      s_row[1] = lnS;
    }
  }
  if (TOP) {
    __syncthreads();
    place_top<kLpThreads>(s_pool, s_n, a.top, t, [&](int r, uint64_t key) {
      write_top(a.out, row, a.top, r, key, s_row[0], s_row[1]);
    });
  }
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
  int stream;     // dlogits is larger than the last-level cache: stores pass it by
};

// Results beyond this many bytes would push one another out of the 256 MB last-level cache
// before anyone reads them.  Stored past it, the gradient of 4095 x 128256 bf16 logits takes
// 322 us instead of 371 (2.1 GB, 6.5 TB/s); results that fit are left in it.
constexpr int64_t kLpCache = (int64_t)256 << 20;

// One workgroup per kLpSlots * kLpThreads * 16 bytes of a row: dz = p (gz - gl - ge (ln p + H))
// + gl [v = t] from the forward's (m, ln S) and H, rounded once; p = exp((z - m) - ln S), so
// that no large number is subtracted from another.
template <int DT>
__global__ __launch_bounds__(kLpThreads) void k_token_logprobs_bwd(LpBwdArgs a) {
  constexpr int EPL = LpT<DT>::EPL, ES = LpT<DT>::ES, U = kLpSlots;
  const long long row = blockIdx.x / a.segs;
  const unsigned seg = blockIdx.x - (unsigned)row * a.segs;
  const char *rp = (const char *)a.logits + row * a.ld * ES;
  char *wp = (char *)a.out + row * a.ld_d * ES;
  const bool stream = a.stream && ((uintptr_t)wp & 15) == 0;
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
      if (stream) __builtin_nontemporal_store(r, (u4 *)(wp + e * ES));
      else store16(wp + e * ES, r);
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

// Splits of a row, the number with the least estimated time (ns): the rounds of one workgroup
// per compute unit that a piece each makes, at 20 bytes a ns and unit, half as much again where
// there is only one workgroup to a unit; the join; and what each workgroup costs by itself.  (Not
// a function of the alternatives, so that their number changes no other result.)  Against 1024
// workgroups or as many as pieces of 4096 allow: 400 rows of 32000 bf16 logits, none: 11.3 -> 8.5
// us, 8: 19.7 -> 15.3 (unsplit); 48 rows of 201088, 5: 17.7 -> 16.4 (ten pieces, not 21); 200
// rows of 128256, 20: 28 either way (five; unsplit 32).
int lp_splits(int64_t N, int64_t V, int dtype) {
  const int64_t most = cd(V, 4096) < kLpMaxSplits ? cd(V, 4096) : kLpMaxSplits;
  if (N < 1 || N > 512) return 1;  // 600 rows of 128256: 31 us whole, 32.8 in halves
  const double row = (double)(V * (dtype == 1 ? 2 : 4)) / 20.0;
  double best = 0.0;
  int s = 1;
  for (int64_t c = 1; c <= most; ++c) {
    const int64_t rounds = (N * c + 255) / 256;
    const double lone = rounds == 1 ? 1.5 : 1.0;
    const double t = lone * (double)rounds / (double)c * row + (c > 1 ? 5000.0 : 0.0) +
                     2.0 * (double)(N * c);
    if (c == 1 || t < best) {
      best = t;
      s = (int)c;
    }
  }
  return s;
}

size_t lp_workspace(int64_t N, int64_t V, int32_t top, int dtype) {
  const int64_t S = lp_splits(N, V, dtype);
  return S == 1 ? 0 : (size_t)(N * S) * (sizeof(LpPart) + 8 * (size_t)top);
}

namespace {
template <int DT, bool TOP>
void run_token_logprobs(const LpArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)(a.N * a.S)), rows((unsigned)a.N);
  if (a.V <= 2048)
    hipLaunchKernelGGL((k_token_logprobs<DT, TOP, 64, 2>), grid, dim3(64), 0, s, a);
  else
    hipLaunchKernelGGL((k_token_logprobs<DT, TOP, kLpThreads, kLpSlots>), grid, dim3(kLpThreads),
                       0, s, a);
  if (a.S > 1)
    hipLaunchKernelGGL((k_token_logprobs_join<DT, TOP>), rows, dim3(kLpThreads), 0, s, a);
}
}  // namespace

hipError_t launch_token_logprobs(int dtype, const void *logits, int64_t ld, const Tokens &tokens,
                                 int64_t N, int64_t V, int32_t top, const LpOut &out, void *ws,
                                 hipStream_t s) {
  if (N <= 0) return hipSuccess;
  int S = lp_splits(N, V, dtype);
  const int64_t per = cd(cd(V, S), 8) * 8;
  S = (int)cd(V, per);
  LpArgs a{logits, ld, N, V, tokens, top, S, per, nullptr, nullptr, out};
  if (S > 1) {
    a.part = (LpPart *)ws;
    a.keys = (uint64_t *)((char *)ws + (size_t)N * S * sizeof(LpPart));
  }
  if (dtype == 1) {
    if (top > 0) run_token_logprobs<1, true>(a, s);
    else run_token_logprobs<1, false>(a, s);
  } else {
    if (top > 0) run_token_logprobs<0, true>(a, s);
    else run_token_logprobs<0, false>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_token_logprobs_bwd(int dtype, const void *logits, int64_t ld,
                                     const Tokens &tokens, int64_t N, int64_t V, const LpGrad &g,
                                     void *dlogits, int64_t ld_d, hipStream_t s) {
  if (N <= 0) return hipSuccess;
  const int64_t epl = dtype == 1 ? 8 : 4;
  LpBwdArgs a{logits, ld, N, V, tokens, g, dlogits, ld_d,
              (unsigned)cd(V, epl * kLpSlots * kLpThreads), N * V * (16 / epl) > kLpCache};
  const dim3 grid((unsigned)(N * a.segs)), block(kLpThreads);
  if (dtype == 1)
    hipLaunchKernelGGL(k_token_logprobs_bwd<1>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(k_token_logprobs_bwd<0>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace kd
