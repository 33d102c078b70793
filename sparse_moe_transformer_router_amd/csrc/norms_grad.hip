// Backward passes of the layer's norms (the pre- and post-norms of the diagram in
// "Porting a 128-expert MoE (Gemma-4 26B-A4B) to AWS Inferentia2", section "The
// architecture: a dual-path FFN nobody warned me about").
//
// A norm n = v r, r = 1 / sqrt(mean(v^2) + eps), y = n g: from d = the gradient of
// y,  d_g = sum_t d n  and, with e = d g,  d_v = r (e - n mean(e n)).
//   before   x -> xd = n g1, xm = n g2 (one n): e = d_xd g1 + d_xm g2; the other
//            gradients of x (the router's, layer_scalar times the output's) are
//            added on the way out.  One pair of row sums: x^2 and e x.
//   behind   s = n(dn) g1 + n(moe) g2, o = n(s) g3, out = (o + x) layer_scalar.
//            Row sums: dn^2 and moe^2; then s^2 and e3 s; then e1 n1 and e2 n2.
// A block takes one row at a time, a thread 8 of its columns (hidden <= 8192), so
// that its sums over tokens (d_g) stay in registers; each block writes them once
// and a second kernel adds the blocks in order.
#include "common.h"
#include "launch.h"

namespace moe {
namespace {

__device__ __forceinline__ void ld8(const float* p, float v[8]) {
  const f32x4* q = reinterpret_cast<const f32x4*>(p);
  const f32x4 a = q[0], b = q[1];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}
__device__ __forceinline__ void ld8(const bf16* p, float v[8]) {
  const bf16x8 b = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)b[j];
}
__device__ __forceinline__ void st8(float* p, const float v[8]) {
  f32x4* q = reinterpret_cast<f32x4*>(p);
  q[0] = f32x4{v[0], v[1], v[2], v[3]};
  q[1] = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void st8(bf16* p, const float v[8]) {
  bf16x8 b;
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = (bf16)v[j];
  *reinterpret_cast<bf16x8*>(p) = b;
}

// Sums of a and b over the block, to every thread.  red: 2 x 16 floats that no
// thread still reads from an earlier call (callers alternate two of them).
__device__ __forceinline__ void block_sum2(float& a, float& b, float* red) {
  a = wave_sum(a);
  b = wave_sum(b);
  const int wave = threadIdx.x / kWave, nw = blockDim.x / kWave;
  if (lane_id() == 0) {
    red[wave] = a;
    red[16 + wave] = b;
  }
  __syncthreads();
  a = b = 0.0f;
  for (int w = 0; w < nw; ++w) {
    a += red[w];
    b += red[16 + w];
  }
}

template <typename XT>
__global__ __launch_bounds__(1024) void pre_grad_kernel(
    int T, int H, float eps, float scalar, const XT* __restrict__ x, const float* __restrict__ g1,
    const float* __restrict__ g2, const uint8_t* __restrict__ mask, const XT* __restrict__ d_xd,
    const XT* __restrict__ d_xm, const XT* __restrict__ d_add, const XT* __restrict__ d_out,
    XT* __restrict__ d_x, float* __restrict__ part) {
  __shared__ float red[2][32];
  const int c = threadIdx.x * 8;
  const bool on = c < H;
  float w1[8] = {}, w2[8] = {}, s1[8] = {}, s2[8] = {};
  if (on) {
    ld8(g1 + c, w1);
    ld8(g2 + c, w2);
  }
  int flip = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const size_t at = (size_t)t * H + c;
    if (mask && !mask[t]) {  // uniform over the block
      const float z[8] = {};
      if (on) st8(d_x + at, z);
      continue;
    }
    float v[8] = {}, a[8] = {}, b[8] = {}, o[8] = {}, ss = 0.0f, es = 0.0f;
    if (on) {
      ld8(x + at, v);
      ld8(d_xd + at, a);
      ld8(d_xm + at, b);
      if (d_out) ld8(d_out + at, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] *= scalar;
      if (d_add) {
        float z[8];
        ld8(d_add + at, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += z[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ss += v[j] * v[j];
      es += (a[j] * w1[j] + b[j] * w2[j]) * v[j];
    }
    block_sum2(ss, es, red[flip]);
    flip ^= 1;
    const float r = 1.0f / sqrtf(ss / (float)H + eps);
    const float m = r * es / (float)H;  // mean(e n)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float n = v[j] * r;
      s1[j] += a[j] * n;
      s2[j] += b[j] * n;
      o[j] += r * (a[j] * w1[j] + b[j] * w2[j] - n * m);
    }
    if (on) st8(d_x + at, o);
  }
  if (on) {
    st8(part + (size_t)blockIdx.x * 2 * H + c, s1);
    st8(part + ((size_t)blockIdx.x * 2 + 1) * H + c, s2);
  }
}

template <typename XT, typename YT>
__global__ __launch_bounds__(1024) void post_grad_kernel(
    int T, int H, float eps, float scalar, const XT* __restrict__ x, const YT* __restrict__ dn,
    const YT* __restrict__ moe_sum, const float* __restrict__ g1, const float* __restrict__ g2,
    const float* __restrict__ g3, const uint8_t* __restrict__ mask, const XT* __restrict__ d_out,
    XT* __restrict__ d_dn, XT* __restrict__ d_moe, float* __restrict__ part,
    double* __restrict__ part_scalar) {
  __shared__ float red[2][32];
  __shared__ double dred[16];
  const int c = threadIdx.x * 8;
  const bool on = c < H;
  float w1[8] = {}, w2[8] = {}, w3[8] = {}, s1[8] = {}, s2[8] = {}, s3[8] = {};
  double ds = 0.0;
  if (on) {
    ld8(g1 + c, w1);
    ld8(g2 + c, w2);
    ld8(g3 + c, w3);
  }
  const float inv = 1.0f / (float)H;
  int flip = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const size_t at = (size_t)t * H + c;
    if (mask && !mask[t]) {
      const float z[8] = {};
      if (on) {
        st8(d_dn + at, z);
        st8(d_moe + at, z);
      }
      continue;
    }
    float a[8] = {}, b[8] = {}, d[8] = {}, xv[8] = {};
    if (on) {
      ld8(dn + at, a);
      ld8(moe_sum + at, b);
      ld8(d_out + at, d);
      if (part_scalar) ld8(x + at, xv);
    }
    float sa = 0.0f, sb = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sa += a[j] * a[j];
      sb += b[j] * b[j];
    }
    block_sum2(sa, sb, red[flip]);
    flip ^= 1;
    const float r1 = 1.0f / sqrtf(sa * inv + eps), r2 = 1.0f / sqrtf(sb * inv + eps);
    float s[8], e3[8], ss = 0.0f, es = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] *= r1;  // n1, n2 from here on
      b[j] *= r2;
      s[j] = a[j] * w1[j] + b[j] * w2[j];
      e3[j] = d[j] * scalar * w3[j];
      ss += s[j] * s[j];
      es += e3[j] * s[j];
    }
    block_sum2(ss, es, red[flip]);
    flip ^= 1;
    const float r3 = 1.0f / sqrtf(ss * inv + eps), m3 = r3 * es * inv;
    float ea = 0.0f, eb = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float n3 = s[j] * r3;
      s3[j] += d[j] * scalar * n3;
      if (part_scalar) ds += (double)d[j] * (double)(n3 * w3[j] + xv[j]);
      const float dsj = r3 * (e3[j] - n3 * m3);
      s1[j] += dsj * a[j];
      s2[j] += dsj * b[j];
      s[j] = dsj;
      ea += dsj * w1[j] * a[j];
      eb += dsj * w2[j] * b[j];
    }
    block_sum2(ea, eb, red[flip]);
    flip ^= 1;
    const float m1 = ea * inv, m2 = eb * inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = r1 * (s[j] * w1[j] - a[j] * m1);
      b[j] = r2 * (s[j] * w2[j] - b[j] * m2);
    }
    if (on) {
      st8(d_dn + at, a);
      st8(d_moe + at, b);
    }
  }
  if (on) {
    float* p = part + (size_t)blockIdx.x * 3 * H + c;
    st8(p, s1);
    st8(p + H, s2);
    st8(p + 2 * (size_t)H, s3);
  }
  if (part_scalar) {
    ds = wave_sum(ds);
    if (lane_id() == 0) dred[threadIdx.x / kWave] = ds;
    __syncthreads();
    if (threadIdx.x == 0) {
      double v = 0.0;
      for (int w = 0; w < (int)blockDim.x / kWave; ++w) v += dred[w];
      part_scalar[blockIdx.x] = v;
    }
  }
}

// out_i[c] = sum over blocks of part[block][i][c], in order within a lane's run of
// blocks, the 16 runs in order.  A block takes 16 columns of n arrays end to end.
__global__ __launch_bounds__(256) void sum_parts_kernel(int nb, int n, int H,
                                                        const float* __restrict__ part,
                                                        float* o1, float* o2, float* o3,
                                                        const double* __restrict__ part_scalar,
                                                        float* d_scalar) {
  __shared__ float red[16][17];
  const int tc = threadIdx.x % 16, tr = threadIdx.x / 16;
  if ((int)blockIdx.x == n * H / 16) {  // the block past the columns: the scalar
    __shared__ double dred[256];
    double v = 0.0;
    for (int b = threadIdx.x; b < nb; b += 256) v += part_scalar[b];
    dred[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      v = 0.0;
      for (int i = 0; i < 256; ++i) v += dred[i];
      *d_scalar = (float)v;
    }
    return;
  }
  const int col = blockIdx.x * 16 + tc;
  float v = 0.0f;
  for (int b = tr; b < nb; b += 16) v += part[(size_t)b * n * H + col];
  red[tr][tc] = v;
  __syncthreads();
  if (tr == 0) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += red[i][tc];
    const int a = col / H, cc = col % H;
    (a == 0 ? o1 : a == 1 ? o2 : o3)[cc] = v;
  }
}

int threads_of(int H) { return (H / 8 + kWave - 1) / kWave * kWave; }

}  // namespace

int norms_grad_blocks(int T) { return T < 512 ? T : 512; }

hipError_t launch_pre_norms_grad(const PreNormGradArgs& a, hipStream_t s) {
  const int nb = norms_grad_blocks(a.T);
  if (nb > 0) {
    if (a.bf16)
      hipLaunchKernelGGL(pre_grad_kernel<bf16>, dim3(nb), dim3(threads_of(a.H)), 0, s, a.T, a.H,
                         a.eps, a.scalar, static_cast<const bf16*>(a.x), a.g1, a.g2, a.mask,
                         static_cast<const bf16*>(a.d_xd), static_cast<const bf16*>(a.d_xm),
                         static_cast<const bf16*>(a.d_add), static_cast<const bf16*>(a.d_out),
                         static_cast<bf16*>(a.d_x), a.ws_part);
    else
      hipLaunchKernelGGL(pre_grad_kernel<float>, dim3(nb), dim3(threads_of(a.H)), 0, s, a.T, a.H,
                         a.eps, a.scalar, static_cast<const float*>(a.x), a.g1, a.g2, a.mask,
                         static_cast<const float*>(a.d_xd), static_cast<const float*>(a.d_xm),
                         static_cast<const float*>(a.d_add), static_cast<const float*>(a.d_out),
                         static_cast<float*>(a.d_x), a.ws_part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sum_parts_kernel, dim3(2 * a.H / 16), dim3(256), 0, s, nb, 2, a.H, a.ws_part,
                     a.d_g1, a.d_g2, nullptr, nullptr, nullptr);
  return hipGetLastError();
}

namespace {

template <typename XT, typename YT>
void launch_post(const PostNormGradArgs& a, int nb, hipStream_t s) {
  hipLaunchKernelGGL((post_grad_kernel<XT, YT>), dim3(nb), dim3(threads_of(a.H)), 0, s, a.T, a.H,
                     a.eps, a.scalar, static_cast<const XT*>(a.x), static_cast<const YT*>(a.dn),
                     static_cast<const YT*>(a.moe_sum), a.g1, a.g2, a.g3, a.mask,
                     static_cast<const XT*>(a.d_out), static_cast<XT*>(a.d_dn),
                     static_cast<XT*>(a.d_moe), a.ws_part, a.d_scalar ? a.ws_scalar : nullptr);
}

}  // namespace

hipError_t launch_post_norms_grad(const PostNormGradArgs& a, hipStream_t s) {
  const int nb = norms_grad_blocks(a.T);
  if (nb > 0) {
    if (!a.bf16) launch_post<float, float>(a, nb, s);
    else if (a.y_bf16) launch_post<bf16, bf16>(a, nb, s);
    else launch_post<bf16, float>(a, nb, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sum_parts_kernel, dim3(3 * a.H / 16 + (a.d_scalar ? 1 : 0)), dim3(256), 0, s,
                     nb, 3, a.H, a.ws_part, a.d_g1, a.d_g2, a.d_g3, a.ws_scalar, a.d_scalar);
  return hipGetLastError();
}

}  // namespace moe
