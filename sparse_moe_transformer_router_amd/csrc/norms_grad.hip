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
// A group of threads takes two rows at a time (one past hidden 4096, and behind the
// branches where the slots are fp32), a thread 8 of their columns (hidden <= 8192), and
// a block as many groups as fit 512 threads (one of up to 1024 past hidden 4096).  The
// sums over tokens (d_g) stay in registers; a block adds its groups' and writes them
// once, and a second kernel adds the blocks in order.  The next rows' loads are issued
// before these are worked on.
// 4096 bf16 tokens of 2816, behind the branches: 138 MB in 46 + 5 us, 3.0 TB/s (one row
// at a time 48 + 5): the three row sums one after another, each a wait for the whole
// group, are not covered by the one block that a CU's registers hold.  With fp32 slots
// 184 MB in 52 + 5 us, all fp32 277 MB in 63 + 5.  Before them 138 MB in 32 + 5 us, 333
// tokens 6.9 + 3.4 us, two launches' latency.  Past hidden 4096 a thread has 128
// registers, and the kernel behind the branches spills 116 to 200 bytes of its rows: 4096
// tokens of 5632, bf16 / fp32 slots / fp32 170 / 216 / 296 us (before them 60 / - / 119).
#include "common.h"
#include "launch.h"

namespace moe {
namespace {

// Blocks of a backward pass at most, one a CU (post-norms at 4096 tokens 48 us, with
// two a CU 52: the blocks' sums are written and read again).
constexpr int kNormsBlocks = 256;

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

// 8 values as loaded.
template <typename T> struct Raw8 { uint4 u[sizeof(T) / 2]; };
template <typename T>
__device__ __forceinline__ Raw8<T> ld_raw(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void widen(const Raw8<T>& r, float v[8]) {
  ld8(reinterpret_cast<const T*>(&r), v);
}

// Sum over the wave, in every lane: within rows of 16 lanes, then across them, on the
// vector unit's own lane moves (a shuffle goes through LDS: six of them in a row took
// a third of a row's time).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf,
                                                        false));
}
__device__ __forceinline__ float wave_total(float v) {
  v = dpp_add<0x111, 0xf>(v);  // row_shr:1, 2, 4, 8
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sums of the N values over the threads of a group (nw waves, this one the w-th of
// group g), to each of them.  red: 16 x N floats that no thread still reads from an
// earlier call (callers alternate two of them).
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float* red, int g, int w, int nw) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = wave_total(v[i]);
    if (lane_id() == 0) red[(g * nw + w) * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int k = 0; k < nw; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += red[(g * nw + k) * N + i];
}

// Adds the groups' sums s (N arrays of H) in order; group 0 writes them to part.
template <int N>
__device__ __forceinline__ void write_sums(float (&s)[N][8], int H, int c, bool on, int g,
                                           int groups, float* lds, float* __restrict__ part) {
  for (int k = 1; k < groups; ++k) {
    __syncthreads();
    if (g == k && on)
#pragma unroll
      for (int i = 0; i < N; ++i) st8(lds + i * H + c, s[i]);
    __syncthreads();
    if (g == 0 && on)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v[8];
        ld8(lds + i * H + c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += v[j];
      }
  }
  if (g == 0 && on)
#pragma unroll
    for (int i = 0; i < N; ++i) st8(part + i * H + c, s[i]);
}

template <typename XT, int MAXT>
__global__ __launch_bounds__(MAXT) void pre_grad_kernel(
    int T, int H, int groups, float eps, float scalar, const XT* x,
    const float* __restrict__ g1, const float* __restrict__ g2, const uint8_t* __restrict__ mask,
    const XT* d_xd, const XT* d_xm, const XT* d_add,
    const XT* d_out, XT* d_x, float* __restrict__ part) {
  constexpr int R = MAXT > 512 ? 1 : 2;  // rows that a group works on at a time
  extern __shared__ __align__(16) float lds[];
  __shared__ __align__(16) float red[2][2 * R * 16];
  const int nt = blockDim.x / groups, nw = nt / kWave;  // threads, waves a group
  const int g = threadIdx.x / nt, c = threadIdx.x % nt * 8, w = threadIdx.x % nt / kWave;
  const bool on = c < H;
  float w1[8] = {}, w2[8] = {}, s[2][8] = {};
  if (on) {
    ld8(g1 + c, w1);
    ld8(g2 + c, w2);
  }
  const int step = gridDim.x * groups * R;
  auto live = [&](int t) { return on && t < T && !(mask && !mask[t]); };
  struct Row { Raw8<XT> x, a, b, z, o; } next[R];
  auto load = [&](int t, Row& r) {
    if (!live(t)) return;
    const size_t at = (size_t)t * H + c;
    r.x = ld_raw(x + at);
    r.a = ld_raw(d_xd + at);
    r.b = ld_raw(d_xm + at);
    if (d_add) r.z = ld_raw(d_add + at);
    if (d_out) r.o = ld_raw(d_out + at);
  };
  int flip = 0;
  const int mine = (blockIdx.x * groups + g) * R;
#pragma unroll
  for (int i = 0; i < R; ++i) load(mine + i, next[i]);
  for (int t0 = blockIdx.x * groups * R; t0 < T; t0 += step) {  // the same for every group
    const int t = t0 + g * R;
    float v[R][8], a[R][8], b[R][8], o[R][8], sum[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = a[i][j] = b[i][j] = o[i][j] = 0.0f;
      if (live(t + i)) {
        widen(next[i].x, v[i]);
        widen(next[i].a, a[i]);
        widen(next[i].b, b[i]);
        if (d_out) widen(next[i].o, o[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[i][j] *= scalar;
        if (d_add) {
          float z[8];
          widen(next[i].z, z);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[i][j] += z[j];
        }
      }
      load(t + step + i, next[i]);
      sum[2 * i] = sum[2 * i + 1] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum[2 * i] += v[i][j] * v[i][j];
        sum[2 * i + 1] += (a[i][j] * w1[j] + b[i][j] * w2[j]) * v[i][j];
      }
    }
    group_sums(sum, red[flip], g, w, nw);
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float r = 1.0f / sqrtf(sum[2 * i] / (float)H + eps);
      const float m = r * sum[2 * i + 1] / (float)H;  // mean(e n)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = v[i][j] * r;
        s[0][j] += a[i][j] * n;
        s[1][j] += b[i][j] * n;
        o[i][j] += r * (a[i][j] * w1[j] + b[i][j] * w2[j] - n * m);
      }
      // zeros where the token does not count
      if (on && t + i < T) st8(d_x + (size_t)(t + i) * H + c, o[i]);
    }
  }
  write_sums<2>(s, H, c, on, g, groups, lds, part + (size_t)blockIdx.x * 2 * H);
}

// Rows that a group of post_grad_kernel works on at a time.  Two of fp32 slots are more
// than its registers hold (60 and 124 bytes a thread spilled with bf16 and fp32
// activations): 4096 tokens of 2816, one / two rows, bf16 slots 48.4 / 46.0 us, fp32 slots
// 51.9 / 65.8, all fp32 63.0 / 105.
template <typename YT>
__host__ __device__ constexpr int post_rows(int threads) {
  return threads > 512 || sizeof(YT) > 2 ? 1 : 2;
}

template <typename XT, typename YT, int MAXT>
__global__ __launch_bounds__(MAXT) void post_grad_kernel(
    int T, int H, int groups, float eps, float scalar, const XT* x,
    const YT* dn, const YT* moe_sum, const float* __restrict__ g1,
    const float* __restrict__ g2, const float* __restrict__ g3, const uint8_t* __restrict__ mask,
    const XT* d_out, XT* d_dn, XT* d_moe,
    float* __restrict__ part, double* __restrict__ part_scalar) {
  constexpr int R = post_rows<YT>(MAXT);
  extern __shared__ __align__(16) float lds[];
  __shared__ __align__(16) float red[2][2 * R * 16];
  __shared__ double dred[16];
  const int nt = blockDim.x / groups, nw = nt / kWave;
  const int g = threadIdx.x / nt, c = threadIdx.x % nt * 8, w = threadIdx.x % nt / kWave;
  const bool on = c < H;
  float w1[8] = {}, w2[8] = {}, w3[8] = {}, sg[3][8] = {};
  double ds = 0.0;
  if (on) {
    ld8(g1 + c, w1);
    ld8(g2 + c, w2);
    ld8(g3 + c, w3);
  }
  const float inv = 1.0f / (float)H;
  const int step = gridDim.x * groups * R;
  auto live = [&](int t) { return on && t < T && !(mask && !mask[t]); };
  struct Row { Raw8<YT> a, b; Raw8<XT> d, x; } next[R];
  auto load = [&](int t, Row& r) {
    if (!live(t)) return;
    const size_t at = (size_t)t * H + c;
    r.a = ld_raw(dn + at);
    r.b = ld_raw(moe_sum + at);
    r.d = ld_raw(d_out + at);
    if (part_scalar) r.x = ld_raw(x + at);
  };
  int flip = 0;
  const int mine = (blockIdx.x * groups + g) * R;
#pragma unroll
  for (int i = 0; i < R; ++i) load(mine + i, next[i]);
  for (int t0 = blockIdx.x * groups * R; t0 < T; t0 += step) {
    const int t = t0 + g * R;
    float a[R][8], b[R][8], d[R][8], xv[R][8], s[R][8], sum[2 * R], r1[R], r2[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) a[i][j] = b[i][j] = d[i][j] = xv[i][j] = 0.0f;
      if (live(t + i)) {
        widen(next[i].a, a[i]);
        widen(next[i].b, b[i]);
        widen(next[i].d, d[i]);
        if (part_scalar) widen(next[i].x, xv[i]);
      }
      load(t + step + i, next[i]);
      sum[2 * i] = sum[2 * i + 1] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum[2 * i] += a[i][j] * a[i][j];
        sum[2 * i + 1] += b[i][j] * b[i][j];
      }
    }
    group_sums(sum, red[flip], g, w, nw);
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      r1[i] = 1.0f / sqrtf(sum[2 * i] * inv + eps);
      r2[i] = 1.0f / sqrtf(sum[2 * i + 1] * inv + eps);
      sum[2 * i] = sum[2 * i + 1] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[i][j] *= r1[i];  // n1, n2 from here on
        b[i][j] *= r2[i];
        s[i][j] = a[i][j] * w1[j] + b[i][j] * w2[j];
        sum[2 * i] += s[i][j] * s[i][j];
        sum[2 * i + 1] += d[i][j] * w3[j] * s[i][j];
      }
    }
    group_sums(sum, red[flip], g, w, nw);
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float r3 = 1.0f / sqrtf(sum[2 * i] * inv + eps), m3 = r3 * sum[2 * i + 1] * inv;
      const float rs = r3 * scalar;
      float row = 0.0f;  // of 8 products; the rows add up in fp64
      sum[2 * i] = sum[2 * i + 1] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n3 = s[i][j] * r3;
        sg[2][j] += d[i][j] * n3;
        row += d[i][j] * (n3 * w3[j] + xv[i][j]);
        const float dsj = rs * (d[i][j] * w3[j] - n3 * m3);
        sg[0][j] += dsj * a[i][j];
        sg[1][j] += dsj * b[i][j];
        s[i][j] = dsj * w1[j];  // e1, and e2 in d's place
        d[i][j] = dsj * w2[j];
        sum[2 * i] += s[i][j] * a[i][j];
        sum[2 * i + 1] += d[i][j] * b[i][j];
      }
      ds += (double)row;
    }
    group_sums(sum, red[flip], g, w, nw);
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float m1 = sum[2 * i] * inv, m2 = sum[2 * i + 1] * inv;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[i][j] = r1[i] * (s[i][j] - a[i][j] * m1);
        b[i][j] = r2[i] * (d[i][j] - b[i][j] * m2);
      }
      if (on && t + i < T) {
        st8(d_dn + (size_t)(t + i) * H + c, a[i]);
        st8(d_moe + (size_t)(t + i) * H + c, b[i]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sg[2][j] *= scalar;
  write_sums<3>(sg, H, c, on, g, groups, lds, part + (size_t)blockIdx.x * 3 * H);
  if (part_scalar) {
    ds = wave_sum(ds);
    if (lane_id() == 0) dred[threadIdx.x / kWave] = ds;
    __syncthreads();
    if (threadIdx.x == 0) {
      double v = 0.0;
      for (int i = 0; i < (int)blockDim.x / kWave; ++i) v += dred[i];
      part_scalar[blockIdx.x] = v;
    }
  }
}

// out_i[c] = sum over blocks of part[block][i][c]: 16 lanes' runs of blocks, each in
// order, added in order.  A block takes 64 columns of the n arrays end to end (H is a
// multiple of 64); the one past the columns adds the scalar's parts.
__global__ __launch_bounds__(1024) void sum_parts_kernel(int nb, int n, int H,
                                                         const float* __restrict__ part,
                                                         float* o1, float* o2, float* o3,
                                                         const double* __restrict__ part_scalar,
                                                         float* d_scalar) {
  const int tc = threadIdx.x % 64, tr = threadIdx.x / 64;
  if ((int)blockIdx.x == n * H / 64) {
    double v = 0.0;
    if (threadIdx.x < 64) {
      for (int b = threadIdx.x; b < nb; b += 64) v += part_scalar[b];
      v = wave_sum(v);
      if (threadIdx.x == 0) *d_scalar = (float)v;
    }
    return;
  }
  __shared__ float red[16][64];
  const int col = blockIdx.x * 64 + tc;
  const float* p = part + col;
  float v = 0.0f;
#pragma unroll 8
  for (int b = tr; b < nb; b += 16) v += p[(size_t)b * n * H];
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

// Threads of a row's group, groups of a block, LDS of a block that adds n arrays.
int threads_of(int H) { return (H / 8 + kWave - 1) / kWave * kWave; }
int groups_of(int H) { return threads_of(H) > 512 ? 1 : 512 / threads_of(H); }
size_t lds_of(int H, int n) { return groups_of(H) > 1 ? (size_t)n * H * 4 : 0; }
int blocks_of(int T, int H, int rows) {  // of groups that take so many rows at a time
  const int n = groups_of(H) * rows, b = (T + n - 1) / n;
  return b < kNormsBlocks ? b : kNormsBlocks;
}
int pre_blocks(int T, int H) { return blocks_of(T, H, threads_of(H) > 512 ? 1 : 2); }
int post_blocks(int T, int H, bool y_bf16) {
  return blocks_of(T, H, y_bf16 ? post_rows<bf16>(threads_of(H)) : post_rows<float>(threads_of(H)));
}

}  // namespace

int norms_grad_blocks(int T, int H, bool y_bf16) {
  const int a = pre_blocks(T, H), b = post_blocks(T, H, y_bf16);
  return a > b ? a : b;
}

namespace {

template <typename XT>
void launch_pre(const PreNormGradArgs& a, int nb, hipStream_t s) {
  auto kf = threads_of(a.H) > 512 ? pre_grad_kernel<XT, 1024> : pre_grad_kernel<XT, 512>;
  hipLaunchKernelGGL(kf, dim3(nb), dim3(threads_of(a.H) * groups_of(a.H)),
                     lds_of(a.H, 2), s, a.T, a.H, groups_of(a.H), a.eps, a.scalar,
                     static_cast<const XT*>(a.x), a.g1, a.g2, a.mask,
                     static_cast<const XT*>(a.d_xd), static_cast<const XT*>(a.d_xm),
                     static_cast<const XT*>(a.d_add), static_cast<const XT*>(a.d_out),
                     static_cast<XT*>(a.d_x), a.ws_part);
}

template <typename XT, typename YT>
void launch_post(const PostNormGradArgs& a, int nb, hipStream_t s) {
  auto kf = threads_of(a.H) > 512 ? post_grad_kernel<XT, YT, 1024> : post_grad_kernel<XT, YT, 512>;
  hipLaunchKernelGGL(kf, dim3(nb),
                     dim3(threads_of(a.H) * groups_of(a.H)), lds_of(a.H, 3), s, a.T, a.H,
                     groups_of(a.H), a.eps, a.scalar, static_cast<const XT*>(a.x),
                     static_cast<const YT*>(a.dn), static_cast<const YT*>(a.moe_sum), a.g1, a.g2,
                     a.g3, a.mask, static_cast<const XT*>(a.d_out), static_cast<XT*>(a.d_dn),
                     static_cast<XT*>(a.d_moe), a.ws_part, a.d_scalar ? a.ws_scalar : nullptr);
}

}  // namespace

hipError_t launch_pre_norms_grad(const PreNormGradArgs& a, hipStream_t s) {
  const int nb = pre_blocks(a.T, a.H);
  if (nb > 0) {
    if (a.bf16) launch_pre<bf16>(a, nb, s);
    else launch_pre<float>(a, nb, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sum_parts_kernel, dim3(2 * a.H / 64), dim3(1024), 0, s, nb, 2, a.H, a.ws_part,
                     a.d_g1, a.d_g2, nullptr, nullptr, nullptr);
  return hipGetLastError();
}

hipError_t launch_post_norms_grad(const PostNormGradArgs& a, hipStream_t s) {
  const int nb = post_blocks(a.T, a.H, a.bf16 && a.y_bf16);
  if (nb > 0) {
    if (!a.bf16) launch_post<float, float>(a, nb, s);
    else if (a.y_bf16) launch_post<bf16, bf16>(a, nb, s);
    else launch_post<bf16, float>(a, nb, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sum_parts_kernel, dim3(3 * a.H / 64 + (a.d_scalar ? 1 : 0)), dim3(1024), 0, s,
                     nb, 3, a.H, a.ws_part, a.d_g1, a.d_g2, a.d_g3, a.ws_scalar, a.d_scalar);
  return hipGetLastError();
}

}  // namespace moe
