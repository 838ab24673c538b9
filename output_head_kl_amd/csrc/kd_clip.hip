// The global norm of many gradient tensors, and clipping to a largest norm.
//
// norm = sqrt(sum over all tensors of sum g^2); where norm > max_norm every element is
// multiplied by max_norm / norm.  Two passes over memory are unavoidable (no element can be
// scaled before the last one is summed): 12 bytes per float32 element in place, 2 launches.
//  * k_sqsum: one workgroup per chunk of a tensor sums its squares in float64 (a square of a
//    float32 neither overflows nor vanishes there) and stores one partial;
//  * k_clip: every workgroup adds up the partials in the same fixed order, so all agree on
//    the scale bit for bit without a third launch between, then scales its chunk.  It takes
//    the chunks in reverse order: the last ones read are still in the last-level cache.
// The tensors' addresses travel in the kernel arguments, a table of kTab at a time, so that
// nothing is copied to the device and a recorded graph holds its own table.
//
// Bound by memory: 420 million float32 elements in place (1.68 GB) take 290 us to sum (5.8
// TB/s) and 660 us to scale (5.1 TB/s, read and write); 48 tensors of 3 million elements in
// all take 12 us on the GPU, less than the host needs to pass them.
#include "kd_ops.h"

#include <cstdint>
#include <cstring>

namespace kd {
namespace {

constexpr int kThreads = 256, kTab = 96, kU = 4;
typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));

struct ClipTab {
  const char *in[kTab];
  char *out[kTab];
  long long n[kTab];
  unsigned first[kTab + 1];  // first chunk of each tensor, and the end
  unsigned char bf16[kTab];
  int count;
  int stream;                // more is written than the last-level cache holds: pass it by
  long long chunk;           // elements, a multiple of 8 * kThreads * kU
};
static_assert(sizeof(ClipTab) < 3500, "kernel arguments stay below 4 KB");

// The chunk's tensor: the last one whose first chunk is not past it.
__device__ __forceinline__ int tab_find(const ClipTab &t, unsigned b) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double x, double *s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  double r = s[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) r += s[i];
  return r;
}

// f(element index, 16 raw bytes, elements in them) over [e0, end) of a tensor.
template <int BF16, class F>
__device__ __forceinline__ void each_group(const char *p, long long e0, long long end, F f) {
  constexpr int EPL = BF16 ? 8 : 4, ES = BF16 ? 2 : 4;
  for (long long e = e0 + threadIdx.x * EPL; e < end; e += (long long)kThreads * kU * EPL) {
    u4 r[kU];
    const long long last = e + (long long)(kU - 1) * kThreads * EPL;
    if (last + EPL <= end) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        __builtin_memcpy(&r[u], p + (e + (long long)u * kThreads * EPL) * ES, 16);
#pragma unroll
      for (int u = 0; u < kU; ++u) f(e + (long long)u * kThreads * EPL, r[u], EPL);
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const long long q = e + (long long)u * kThreads * EPL;
        if (q >= end) break;
        if (q + EPL <= end) {
          __builtin_memcpy(&r[u], p + q * ES, 16);
          f(q, r[u], EPL);
        } else {
          r[u] = u4{0u, 0u, 0u, 0u};
          const int n = (int)(end - q);
#pragma unroll
          for (int j = 0; j < EPL; ++j)
            if (j < n) {
              if (BF16) r[u][j >> 1] |= (unsigned)((const unsigned short *)p)[q + j] << (16 * (j & 1));
              else r[u][j] = ((const unsigned *)p)[q + j];
            }
          f(q, r[u], n);
        }
      }
    }
  }
}

template <int BF16>
__device__ __forceinline__ double square_sum(const char *p, long long e0, long long end) {
  double acc[2] = {0.0, 0.0};
  each_group<BF16>(p, e0, end, [&](long long, u4 r, int) {  // elements past the end are 0
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (BF16) {
        const double a = (double)__uint_as_float(r[j] << 16);
        const double b = (double)__uint_as_float(r[j] & 0xFFFF0000u);
        acc[0] = fma(a, a, acc[0]);
        acc[1] = fma(b, b, acc[1]);
      } else {
        const double a = (double)__uint_as_float(r[j]);
        acc[j & 1] = fma(a, a, acc[j & 1]);
      }
    }
  });
  return acc[0] + acc[1];
}

__global__ __launch_bounds__(kThreads) void k_sqsum(ClipTab t, double *part) {
  __shared__ double s[kThreads / 64];
  const unsigned b = blockIdx.x;
  const int i = tab_find(t, b);
  const long long e0 = (long long)(b - t.first[i]) * t.chunk;
  const long long end = e0 + t.chunk < t.n[i] ? e0 + t.chunk : t.n[i];
  const double x = t.bf16[i] ? square_sum<1>(t.in[i], e0, end) : square_sum<0>(t.in[i], e0, end);
  const double r = block_sum(x, s);
  if (threadIdx.x == 0) part[b] = r;
}

// The norm of all partials, the same in every workgroup.
__device__ __forceinline__ float norm_of(const double *part, long long npart, double *s) {
  double x = 0.0;
  for (long long i = threadIdx.x; i < npart; i += kThreads) x += part[i];
  return (float)sqrt(block_sum(x, s));
}

__global__ __launch_bounds__(kThreads) void k_norm(const double *part, long long npart, float *norm) {
  __shared__ double s[kThreads / 64];
  const float r = norm_of(part, npart, s);
  if (threadIdx.x == 0) *norm = r;
}

template <int BF16>
__device__ __forceinline__ void scale_chunk(const char *in, char *out, long long e0, long long end,
                                            float s, bool stream) {
  constexpr int ES = BF16 ? 2 : 4;
  stream = stream && ((uintptr_t)out & 15) == 0;
  each_group<BF16>(in, e0, end, [&](long long e, u4 r, int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (BF16)  // one rounding, to nearest even
        r[j] = __builtin_bit_cast(unsigned, __builtin_convertvector(
                                                f2{__uint_as_float(r[j] << 16) * s,
                                                   __uint_as_float(r[j] & 0xFFFF0000u) * s}, b2));
      else
        r[j] = __float_as_uint(__uint_as_float(r[j]) * s);
    }
    if (n == (BF16 ? 8 : 4)) {
      if (stream) __builtin_nontemporal_store(r, (u4 *)(out + e * ES));
      else __builtin_memcpy(out + e * ES, &r, 16);
    } else {
#pragma unroll
      for (int j = 0; j < (BF16 ? 8 : 4); ++j)
        if (j < n) {
          if (BF16) ((unsigned short *)out)[e + j] = (unsigned short)(r[j >> 1] >> (16 * (j & 1)));
          else ((unsigned *)out)[e + j] = r[j & 3];
        }
    }
  });
}

__global__ __launch_bounds__(kThreads) void k_clip(ClipTab t, const double *part, long long npart,
                                                   float max_norm, float *norm) {
  __shared__ double s[kThreads / 64];
  const float r = norm_of(part, npart, s);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = r;
  const float scale = r > max_norm && r < INFINITY ? (float)((double)max_norm / (double)r) : 1.f;
  const unsigned b = gridDim.x - 1 - blockIdx.x;
  const int i = tab_find(t, b);
  if (scale == 1.f && t.in[i] == t.out[i]) return;  // nothing changes in place
  const long long e0 = (long long)(b - t.first[i]) * t.chunk;
  const long long end = e0 + t.chunk < t.n[i] ? e0 + t.chunk : t.n[i];
  if (t.bf16[i]) scale_chunk<1>(t.in[i], t.out[i], e0, end, scale, t.stream);
  else scale_chunk<0>(t.in[i], t.out[i], e0, end, scale, t.stream);
}

// Chunks of at least 8192 elements, and longer ones once there would be more than about
// 4096: every workgroup of k_clip reads all partials.
int64_t chunk_of(const int64_t *numel, int32_t n) {
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) total += numel[i];
  const int64_t unit = 8 * kThreads * kU, c = (total / 4096 + unit - 1) / unit * unit;
  return c < unit ? unit : c;
}

}  // namespace

int64_t clip_partials(const int64_t *numel, int32_t n) {
  const int64_t c = chunk_of(numel, n);
  int64_t p = 0;
  for (int32_t i = 0; i < n; ++i) p += (numel[i] + c - 1) / c;
  return p;
}

hipError_t launch_clip_grads(const void *const *grads, void *const *outs, const int64_t *numel,
                             const int32_t *dtypes, int32_t n, bool scale, float max_norm,
                             float *norm, double *part, hipStream_t s) {
  const int64_t chunk = chunk_of(numel, n), npart = clip_partials(numel, n);
  int64_t bytes = 0;
  for (int32_t i = 0; i < n; ++i) bytes += numel[i] * (dtypes[i] == 1 ? 2 : 4);
  for (int pass = 0; pass < (scale && npart > 0 ? 2 : 1); ++pass) {
    int64_t base = 0;
    bool first = true;
    for (int32_t i = 0; i < n;) {
      ClipTab t;
      t.count = 0;
      t.chunk = chunk;
      t.stream = bytes > ((int64_t)256 << 20);
      unsigned blocks = 0;
      for (; i < n && t.count < kTab; ++i) {
        if (numel[i] == 0) continue;
        const int k = t.count++;
        t.in[k] = (const char *)grads[i];
        t.out[k] = outs ? (char *)outs[i] : (char *)const_cast<void *>(grads[i]);
        t.n[k] = numel[i];
        t.first[k] = blocks;
        t.bf16[k] = dtypes[i] == 1;
        blocks += (unsigned)((numel[i] + chunk - 1) / chunk);
      }
      t.first[t.count] = blocks;
      if (blocks == 0) continue;
      if (pass == 0)
        hipLaunchKernelGGL(k_sqsum, dim3(blocks), dim3(kThreads), 0, s, t, part + base);
      else
        hipLaunchKernelGGL(k_clip, dim3(blocks), dim3(kThreads), 0, s, t, (const double *)part,
                           (long long)npart, max_norm, first ? norm : (float *)nullptr);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      first = false;
      base += blocks;
    }
  }
  if (!scale || npart == 0)
    hipLaunchKernelGGL(k_norm, dim3(1), dim3(kThreads), 0, s, (const double *)part,
                       (long long)npart, norm);
  return hipGetLastError();
}

}  // namespace kd
