// Global norm of a list of gradients, and their clipping.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   coef = min(1, max_norm / (norm + 1e-6)),   g <- coef g
//
// Bound by memory: one read of every gradient for the norm; a second read and a
// write for the clipping, which cannot begin before the norm is known.  The list
// of tensors travels in the kernels' arguments (no copy to the device, nothing
// that a captured graph could find changed), kTable of them a launch.  A tensor
// is cut into chunks, dealt out to the blocks in turn; each block
// adds its chunks' squares in fp64 (an fp32 square overflows from 2^64 on and
// vanishes below 2^-75) and writes one partial sum, added in order by a last block:
// results repeat bit for bit.
// A layer's 780M bf16 gradients: the norm 248 us (1.56 GB read, 6.3 TB/s), the
// clipping 572 us (3.12 GB, 5.5 TB/s; a large copy reaches 4.85).
#include "common.h"
#include "launch.h"
#include "moe.h"

namespace moe {
namespace {

constexpr int kTable = 128;              // tensors a launch
// Elements a chunk: few in short lists, for more blocks.  Norm + clipping of 0.38M fp32 /
// 1M / 4M / 16M bf16 elements, 2048: 8.0 / 8.2 / 11.1 / 24.8 us, 16384: 11.4 / 11.0 / 13.2
// / 24.2; 64M: 69 and 60.
constexpr int kChunk = 16384, kSmallChunk = 2048;
constexpr long long kSmallList = 1 << 23;
// Lists whose results go past the caches: from 64 MB of bf16 on, a quarter of the last
// cache.  780M elements: the clipping 572 us (565 through the caches), the next norm 248
// (283).
constexpr long long kPastList = 1 << 25;
constexpr int kThreads = 256;
constexpr int kNormBlocks = 2048;        // blocks of a norm launch at most

struct Table {
  const void* src[kTable];
  void* dst[kTable];
  long long numel[kTable];
  int first[kTable + 1];                 // first chunk of each tensor
  unsigned char src_bf16[kTable], dst_bf16[kTable];
  int n, chunk;                          // tensors; elements a chunk
};
static_assert(sizeof(Table) <= 3968, "kernel arguments");

// Tensor that chunk c belongs to.
__device__ __forceinline__ int find(const Table& t, int c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* __restrict__ p, int n) {
  double s = 0.0;
  constexpr int V = 16 / (int)sizeof(T);
  if (aligned16(p)) {
    const int nv = n / V;
    for (int i = threadIdx.x; i < nv; i += kThreads) {
      T v[V];
      *reinterpret_cast<uint4*>(v) = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const double d = (double)to_f32(v[j]);
        s = fma(d, d, s);
      }
    }
    for (int i = nv * V + threadIdx.x; i < n; i += kThreads) {
      const double d = (double)to_f32(p[i]);
      s = fma(d, d, s);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const double d = (double)to_f32(p[i]);
      s = fma(d, d, s);
    }
  }
  return s;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kThreads / kWave];
  v = wave_sum(v);
  if (lane_id() == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) v += red[w];
  return v;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const Table t, double* __restrict__ part) {
  double s = 0.0;
  for (int c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const int i = find(t, c);
    const long long at = (long long)(c - t.first[i]) * t.chunk;
    const int n = (int)min((long long)t.chunk, t.numel[i] - at);
    if (t.src_bf16[i]) s += chunk_squares(static_cast<const bf16*>(t.src[i]) + at, n);
    else s += chunk_squares(static_cast<const float*>(t.src[i]) + at, n);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void norm_end_kernel(int nparts, float max_norm,
                                                            const double* __restrict__ part,
                                                            float* __restrict__ norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) s += part[i];
  s = block_sum(s);
  if (threadIdx.x == 0) {
    const float v = (float)sqrt(s);
    const float c = max_norm / (v + 1e-6f);
    norm[0] = v;
    norm[1] = c > 1.0f ? 1.0f : c;  // a NaN stays one
  }
}

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

template <bool PAST, typename S, typename D>
__device__ __forceinline__ void chunk_scale(const S* p, D* q, int n, float coef) {
  if (aligned16(p) && aligned16(q)) {
    const int nv = n / 8;
    for (int i = threadIdx.x; i < nv; i += kThreads) {
      S v[8];
      D o[8];
#pragma unroll
      for (int j = 0; j < (int)sizeof(S) / 2; ++j)
        reinterpret_cast<uint4*>(v)[j] = reinterpret_cast<const uint4*>(p + 8 * (size_t)i)[j];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = from_f32<D>(to_f32(v[j]) * coef);
#pragma unroll
      for (int j = 0; j < (int)sizeof(D) / 2; ++j) {
        u32x4* to = reinterpret_cast<u32x4*>(q + 8 * (size_t)i) + j;
        if constexpr (PAST) __builtin_nontemporal_store(reinterpret_cast<u32x4*>(o)[j], to);
        else *to = reinterpret_cast<u32x4*>(o)[j];
      }
    }
    for (int i = nv * 8 + threadIdx.x; i < n; i += kThreads)
      q[i] = from_f32<D>(to_f32(p[i]) * coef);
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) q[i] = from_f32<D>(to_f32(p[i]) * coef);
  }
}

// Chunks from the last to the first: the norm's pass read the last ones last, so
// they are the likeliest to be in the caches still.  PAST: the results go past the
// caches, where they would be written back while a later kernel reads.
template <bool PAST>
__global__ __launch_bounds__(kThreads) void clip_kernel(const Table t,
                                                        const float* __restrict__ norm) {
  const float coef = norm[1];
  const int total = t.first[t.n];
  for (int k = blockIdx.x; k < total; k += gridDim.x) {
    const int c = total - 1 - k, i = find(t, c);
    if (coef == 1.0f && t.dst[i] == t.src[i] && t.src_bf16[i] == t.dst_bf16[i]) continue;
    const long long at = (long long)(c - t.first[i]) * t.chunk;
    const int n = (int)min((long long)t.chunk, t.numel[i] - at);
    if (t.src_bf16[i]) {
      const bf16* p = static_cast<const bf16*>(t.src[i]) + at;
      if (t.dst_bf16[i]) chunk_scale<PAST>(p, static_cast<bf16*>(t.dst[i]) + at, n, coef);
      else chunk_scale<PAST>(p, static_cast<float*>(t.dst[i]) + at, n, coef);
    } else {
      const float* p = static_cast<const float*>(t.src[i]) + at;
      if (t.dst_bf16[i]) chunk_scale<PAST>(p, static_cast<bf16*>(t.dst[i]) + at, n, coef);
      else chunk_scale<PAST>(p, static_cast<float*>(t.dst[i]) + at, n, coef);
    }
  }
}

long long elements(int n, const moe_tensor* t) {
  long long total = 0;
  for (int i = 0; i < n; ++i) total += t[i].numel;
  return total;
}
int chunk_of(long long total) { return total < kSmallList ? kSmallChunk : kChunk; }

// The next tensors of a list, from `at` on, as a launch's table: at most kTable
// tensors with elements (the callers hold them to 2^40 elements, 2^26 chunks).
void fill(Table& tb, int n, const moe_tensor* t, const moe_tensor* out, int chunk, int& at) {
  tb.n = 0;
  tb.first[0] = 0;
  tb.chunk = chunk;
  for (; at < n && tb.n < kTable; ++at) {
    if (t[at].numel == 0) continue;
    const int i = tb.n++;
    tb.src[i] = t[at].data;
    tb.src_bf16[i] = t[at].dtype == MOE_BF16;
    tb.dst[i] = out ? out[at].data : t[at].data;
    tb.dst_bf16[i] = (out ? out : t)[at].dtype == MOE_BF16;
    tb.numel[i] = t[at].numel;
    tb.first[i + 1] = tb.first[i] + (int)((t[at].numel + chunk - 1) / chunk);
  }
}

}  // namespace

long long grad_norm_parts(int n, const moe_tensor* t) {
  const int chunk = chunk_of(elements(n, t));
  long long parts = 0;
  int at = 0;
  while (at < n) {
    Table tb;
    fill(tb, n, t, nullptr, chunk, at);
    parts += tb.first[tb.n] < kNormBlocks ? tb.first[tb.n] : kNormBlocks;
  }
  return parts;
}

hipError_t launch_grad_norm(int n, const moe_tensor* t, float max_norm, float* norm,
                            double* ws_part, hipStream_t s) {
  const int chunk = chunk_of(elements(n, t));
  int parts = 0, at = 0;
  while (at < n) {
    Table tb;
    fill(tb, n, t, nullptr, chunk, at);
    const int blocks = tb.first[tb.n] < kNormBlocks ? tb.first[tb.n] : kNormBlocks;
    if (blocks == 0) continue;
    hipLaunchKernelGGL(norm_kernel, dim3(blocks), dim3(kThreads), 0, s, tb, ws_part + parts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    parts += blocks;
  }
  hipLaunchKernelGGL(norm_end_kernel, dim3(1), dim3(kThreads), 0, s, parts, max_norm, ws_part,
                     norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(int n, const moe_tensor* t, const float* norm, const moe_tensor* out,
                            hipStream_t s) {
  const long long total = elements(n, t);
  const int chunk = chunk_of(total);
  auto kf = total < kPastList ? clip_kernel<false> : clip_kernel<true>;
  int at = 0;
  while (at < n) {
    Table tb;
    fill(tb, n, t, out, chunk, at);
    const int chunks = tb.first[tb.n];
    if (chunks == 0) continue;
    hipLaunchKernelGGL(kf, dim3(chunks < 8192 ? chunks : 8192), dim3(kThreads), 0, s, tb,
                       norm);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
