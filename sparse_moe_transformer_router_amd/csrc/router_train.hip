// Training side of the router (Gemma4TextRouter on the page "Porting a
// 128-expert MoE (Gemma-4 26B-A4B) to AWS Inferentia2", section "The
// architecture: a dual-path FFN nobody warned me about"): the balance loss and
// z-loss of a batch with the tokens each expert received, the loss's gradient
// in the logits, and the backward pass from the gradient of the routing
// weights and logits to the router's input and parameters.
//
// Every sum runs in fp32 in an order fixed by the sizes alone (no
// floating-point atomics), so results repeat bit for bit.  Counts are integers.
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "route_dev.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Reductions over the G = 8, 16, 32 or 64 lanes that share a token; every lane
// of the group gets the result.  Within 16 lanes they are DPP moves (quad
// permutes, then the mirrors of 8 and 16 lanes), past that lane shuffles.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

template <int G, typename F>
__device__ __forceinline__ float group_reduce(float v, F f) {
  static_assert(G == 8 || G == 16 || G == 32 || G == 64, "lanes per token");
  v = f(v, dpp_f32<kDppXor1>(v));
  v = f(v, dpp_f32<kDppXor2>(v));
  v = f(v, dpp_f32<kDppHalfMirror>(v));
  if constexpr (G >= 16) v = f(v, dpp_f32<kDppMirror>(v));
  if constexpr (G >= 32) v = f(v, __shfl_xor(v, 16, kWave));
  if constexpr (G >= 64) v = f(v, __shfl_xor(v, 32, kWave));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<G>(v, [](float a, float b) { return a + b; });
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

// Four consecutive logits e0 .. e0 + 3 of a row; past the last expert -inf,
// whose probability is 0.  VEC: E % 4 == 0, so every row is 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ void load_logits4(const float* __restrict__ row, int e0, int E,
                                             float (&l)[4]) {
  if constexpr (VEC) {
    if (e0 < E) {
      const float4 v = *reinterpret_cast<const float4*>(row + e0);
      l[0] = v.x; l[1] = v.y; l[2] = v.z; l[3] = v.w;
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) l[j] = e0 + j < E ? row[e0 + j] : -INFINITY;
}

// exp(x), x <= 0, on the hardware's power of two: the product's rounding moves the
// result by |x| 2^-24, as much as the rounding of l - max did.
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}

// Softmax numerators of a token's logits: l becomes exp(l - max), z their sum
// over the group, lse the row's log-sum-exp.  A row of -inf only has no
// probability anywhere: z is 0 and inv (1 / z) and lse are 0.
template <int G>
__device__ __forceinline__ void group_softmax(float (&l)[4], float& inv, float& lse) {
  const float top = group_max<G>(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
  const bool none = top == -INFINITY;
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    l[j] = none ? 0.0f : exp_neg(l[j] - top);
    z += l[j];
  }
  z = group_sum<G>(z);
  inv = none ? 0.0f : 1.0f / z;
  lse = none ? 0.0f : top + logf(z);
}

// ---------------------------------------------------------------------------
// Balance loss, first step.  N live tokens (token_mask, or all of them):
//   n_e = slots of live tokens routed to e,  f_e = n_e / (N K),
//   P_e = 1/N sum_t softmax(l_t)_e,          lse_t = log sum_e exp l_te,
//   balance = E sum_e f_e P_e,               z = 1/N sum_t lse_t^2.
// Block b takes tokens [b * span, ...): G lanes a token, four experts a lane,
// kept in registers over the block's tokens, while four more waves count the
// block's slots.  It writes its sums of P_e, its counts, its sum of lse^2 and its
// number of live tokens; the second step adds the blocks in order.  A batch of
// one block's size runs both steps in one launch.
//
// Reads the logits once: 65536 x 128 in 12.6 us (2.8 TB/s; 12 softmax waves a block
// 12.2, 512 blocks 12.0 but a second step of 7.6 us instead of 4.7), 4096 x 128 in
// 5.0 us, 64 in 4.1: there a launch and one round trip to memory.
// ---------------------------------------------------------------------------
constexpr int kBalWaves = 8, kBalCountWaves = 4;  // softmax, counts
constexpr int kBalThreads = (kBalWaves + kBalCountWaves) * kWave;
constexpr int kBalCountThreads = kBalCountWaves * kWave;
constexpr int kBalUnroll = 4;       // tokens a group loads before it adds the first
constexpr int kBalOneBlock = 256;   // tokens that one block takes alone
constexpr int kBalMaxBlocks = 256;  // one block per CU

// loss[4] = {a * balance + b * z, balance, z, N}; mean_p = P.  Called by the
// whole block with the summed values of expert tid (tid < E).
__device__ __forceinline__ void balance_finish(int E, int K, float a, float b, float sum_p,
                                               int count, float sum_z, int live,
                                               float* __restrict__ loss,
                                               int32_t* __restrict__ counts,
                                               float* __restrict__ mean_p, float* red) {
  const int tid = threadIdx.x;
  const float inv = live > 0 ? 1.0f / (float)live : 0.0f;
  float fp = 0.0f;
  if (tid < E) {
    const float p = sum_p * inv;
    counts[tid] = count;
    mean_p[tid] = p;
    fp = ((float)count * (inv / (float)K)) * p;
  }
  fp = wave_sum(fp);  // E <= 256: the first four waves hold terms
  if (lane_id() == 0) red[tid / kWave] = fp;
  __syncthreads();
  if (tid == 0) {
    const float bal = (float)E * (((red[0] + red[1]) + red[2]) + red[3]);
    const float z = sum_z * inv;
    loss[0] = a * bal + b * z;
    loss[1] = bal;
    loss[2] = z;
    loss[3] = (float)live;
  }
}

template <int G, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_partial_kernel(
    int T, int E, int K, int span, const float* __restrict__ logits,
    const int32_t* __restrict__ topk_idx, const uint8_t* __restrict__ mask, float a, float b,
    float* __restrict__ part_p, int32_t* __restrict__ part_n, float* __restrict__ part_z,
    int32_t* __restrict__ part_live, float* __restrict__ loss, int32_t* __restrict__ counts,
    float* __restrict__ mean_p) {
  constexpr int TW = kWave / G;             // tokens per wave
  constexpr int TB = TW * kBalWaves;        // tokens per block and round
  __shared__ float sum_p[kBalWaves * TW][4 * G];
  __shared__ int cnt[kBalCountWaves][kMaxE];
  __shared__ float wave_z[kBalWaves];
  __shared__ int wave_live[kBalWaves];
  __shared__ float red[kBalThreads / kWave];
  const int tid = threadIdx.x, wave = tid / kWave, lane = lane_id();
  const int t0 = blockIdx.x * span, t1 = min(T, t0 + span);
  if (wave >= kBalWaves) {
    // one counter row per wave, cleared and used by that wave alone
    int* mine = cnt[wave - kBalWaves];
    for (int e = lane; e < kMaxE; e += kWave) mine[e] = 0;
    constexpr int U = 8;  // slots a lane loads before it counts the first
    for (int s0 = t0 * K + tid - kBalWaves * kWave; s0 < t1 * K; s0 += U * kBalCountThreads) {
      int e[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u * kBalCountThreads, sc = min(s, t1 * K - 1);
        e[u] = topk_idx[sc];
        on[u] = s < t1 * K && (mask == nullptr || mask[sc / K] != 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (on[u] && (unsigned)e[u] < (unsigned)E) atomicAdd(&mine[e[u]], 1);
    }
  } else {
    const int gl = lane % G, grp = wave * TW + lane / G;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float zsum = 0.0f;
    int live = 0;
    float next[kBalUnroll][4];
    auto load = [&](int t) {
#pragma unroll
      for (int u = 0; u < kBalUnroll; ++u)
        load_logits4<VEC>(logits + (size_t)min(t + u * TB, t1 - 1) * E, 4 * gl, E, next[u]);
    };
    if (t0 + grp < t1) load(t0 + grp);
    for (int t = t0 + grp; t < t1; t += TB * kBalUnroll) {
      float l[kBalUnroll][4];
      bool on[kBalUnroll];
#pragma unroll
      for (int u = 0; u < kBalUnroll; ++u) {
        const int tu = min(t + u * TB, t1 - 1);
        on[u] = t + u * TB < t1 && (mask == nullptr || mask[tu] != 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) l[u][j] = next[u][j];
      }
      if (t + TB * kBalUnroll < t1) load(t + TB * kBalUnroll);
#pragma unroll
      for (int u = 0; u < kBalUnroll; ++u) {
        float inv, lse;
        group_softmax<G>(l[u], inv, lse);
        if (on[u]) {  // a masked row may hold anything
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] += l[u][j] * inv;
          zsum += lse * lse;
          live += 1;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum_p[grp][4 * gl + j] = acc[j];
    // one lane of each group holds its tokens' sum
    zsum = wave_sum(gl == 0 ? zsum : 0.0f);
    live = wave_sum(gl == 0 ? live : 0);
    if (lane == 0) {
      wave_z[wave] = zsum;
      wave_live[wave] = live;
    }
  }
  __syncthreads();
  float p = 0.0f, z = 0.0f;
  int n = 0, nl = 0;
  if (tid < E) {
    for (int w = 0; w < kBalWaves * TW; ++w) p += sum_p[w][tid];
    for (int w = 0; w < kBalCountWaves; ++w) n += cnt[w][tid];
  }
  for (int w = 0; w < kBalWaves; ++w) {
    z += wave_z[w];
    nl += wave_live[w];
  }
  if (gridDim.x == 1) {
    balance_finish(E, K, a, b, p, n, z, nl, loss, counts, mean_p, red);
    return;
  }
  if (tid < E) {
    part_p[(size_t)blockIdx.x * E + tid] = p;
    part_n[(size_t)blockIdx.x * E + tid] = n;
  }
  if (tid == 0) {
    part_z[blockIdx.x] = z;
    part_live[blockIdx.x] = nl;
  }
}

// Second step: one block of 1024 threads adds the blocks' sums; expert e's nb
// values are split over the thread rows, whose sums are added in order.
constexpr int kBalFinThreads = 1024;
__global__ __launch_bounds__(kBalFinThreads) void balance_final_kernel(
    int nb, int E, int K, float a, float b, const float* __restrict__ part_p,
    const int32_t* __restrict__ part_n, const float* __restrict__ part_z,
    const int32_t* __restrict__ part_live, float* __restrict__ loss,
    int32_t* __restrict__ counts, float* __restrict__ mean_p) {
  __shared__ float sp[kBalFinThreads];
  __shared__ int sn[kBalFinThreads];
  __shared__ float wz[kBalFinThreads / kWave];
  __shared__ int wl[kBalFinThreads / kWave];
  __shared__ float red[kBalFinThreads / kWave];
  const int tid = threadIdx.x;
  const int rows = kBalFinThreads / E;  // E <= 256: four or more
  const int e = tid % E, r = tid / E;
  float p = 0.0f;
  int n = 0;
  if (r < rows) {
#pragma unroll 8
    for (int i = r; i < nb; i += rows) {
      p += part_p[(size_t)i * E + e];
      n += part_n[(size_t)i * E + e];
    }
  }
  sp[tid] = p;
  sn[tid] = n;
  float z = tid < nb ? part_z[tid] : 0.0f;  // nb <= kBalMaxBlocks
  int live = tid < nb ? part_live[tid] : 0;
  z = wave_sum(z);
  live = wave_sum(live);
  if (lane_id() == 0) {
    wz[tid / kWave] = z;
    wl[tid / kWave] = live;
  }
  __syncthreads();
  p = 0.0f;
  n = 0;
  if (tid < E)
    for (int i = 0; i < rows; ++i) {
      p += sp[i * E + tid];
      n += sn[i * E + tid];
    }
  z = 0.0f;
  live = 0;
  for (int w = 0; w < kBalMaxBlocks / kWave; ++w) {
    z += wz[w];
    live += wl[w];
  }
  balance_finish(E, K, a, b, p, n, z, live, loss, counts, mean_p, red);
}

// Gradient of g * loss[0] in the logits, g = *d_loss:
//   d l_tj = g [ a E / N p_tj (f_j - sum_e f_e p_te) + 2 b / N lse_t p_tj ],
// 0 for masked tokens and for a row of -inf.  Memory-bound: the logits read
// and the gradient written once; f_e of a lane's four experts in registers
// (65536 x 128: 17.3 us, 3.9 TB/s; 4096: 4.7 us; four tokens a group and step
// instead of two 16.8 and 5.9).
constexpr int kGradUnroll = 2;
template <int G, bool VEC>
__global__ __launch_bounds__(256) void balance_grad_kernel(
    int T, int E, int K, const float* logits, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ counts, const float* __restrict__ loss, float a, float b,
    const float* __restrict__ d_loss, float* d_logits) {  // d_logits may be logits
  constexpr int TB = 256 / G;
  const int gl = threadIdx.x % G, grp = threadIdx.x / G, e0 = 4 * gl;
  const float n = loss[3];
  const float inv_n = n > 0.0f ? 1.0f / n : 0.0f;
  const float up = d_loss[0] * inv_n;
  const float ca = up * a * (float)E, cb = 2.0f * up * b;
  const float fs = inv_n / (float)K;
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = e0 + j < E ? (float)counts[e0 + j] * fs : 0.0f;
  for (int t = blockIdx.x * TB * kGradUnroll + grp; t < T; t += gridDim.x * TB * kGradUnroll) {
    float l[kGradUnroll][4];
    bool on[kGradUnroll];
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      const int tu = min(t + u * TB, T - 1);
      on[u] = mask == nullptr || mask[tu] != 0;
      load_logits4<VEC>(logits + (size_t)tu * E, e0, E, l[u]);
    }
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      float inv, lse;
      group_softmax<G>(l[u], inv, lse);
      float pf = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        l[u][j] *= inv;
        pf += l[u][j] * f[j];
      }
      pf = group_sum<G>(pf);
      float d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        d[j] = on[u] ? l[u][j] * (ca * (f[j] - pf) + cb * lse) : 0.0f;
      if (t + u * TB < T && e0 < E) {
        float* dst = d_logits + (size_t)(t + u * TB) * E + e0;
        if constexpr (VEC) {
          *reinterpret_cast<float4*>(dst) = make_float4(d[0], d[1], d[2], d[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (e0 + j < E) dst[j] = d[j];
        }
      }
    }
  }
}

// Calls go(G, VEC) for E experts.
template <typename F>
void by_group(int E, F go) {
  auto vec = [&](auto g) {
    if (E % 4 == 0) go(g, std::true_type{});
    else go(g, std::false_type{});
  };
  if (E <= 32) vec(std::integral_constant<int, 8>{});
  else if (E <= 64) vec(std::integral_constant<int, 16>{});
  else if (E <= 128) vec(std::integral_constant<int, 32>{});
  else vec(std::integral_constant<int, 64>{});
}

// ---------------------------------------------------------------------------
// Router backward.  With r0 = 1/sqrt(mean x^2 + eps), v = x r0 g (pre-norm)
// or x, r = 1/sqrt(mean v^2 + eps), vhat = v r c, l = W vhat, and the gradient
// dl of the logits, the norm's own terms need no second pass over H: since
// sum_h (c W^T dl)_h v_h = D / r with D = sum_e dl_e l_e,
//   dl' = dl r0 r,   beta = r0^2 r^2 D / H   (r0 = 1 without a pre-norm)
//   G = dl'^T x [E,H],   m_h = sum_e W_eh G_eh
//   dW = G g c,   dc = g m,   dg = c m - g sum_t x^2 beta
//   dx = g c (dl' W) - x beta (g^2 + eps)    with a pre-norm
//   dx =   c (dl' W) - x beta                without (g = 1)
// (the pre-norm's projection, sum_h g dv x, is D r^2 eps / r0).
//
// First kernel, a wave per token: the routing weights' gradient to the
// logits (q = softmax over the K picked, dl_k = q_k (d_k - sum_j q_j d_j) with
// d_k = d_topk_w_k * per_expert_scale), plus the given d_logits; the two
// norms; dl', beta, and the block's sums of d_topk_w_k q_k per expert.  Bound by
// the latency of a token's chain (picks, logits, x, sums over 64 lanes): 9 us for
// 301 tokens, 12 for 4096 of 2816 bf16 values (1.9 TB/s).
// ---------------------------------------------------------------------------
constexpr int kRgRowWaves = 16;  // a token each

__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Eight values as loaded.
template <typename XT> struct Piece;
template <> struct Piece<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Piece<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// One token's share, by a wave: dl (experts lane + 64 j) scaled by r0 r, beta,
// and d_topk_w_k q_k added to dpes.  A masked token gives zeros.
template <typename XT>
__device__ __forceinline__ void router_grad_token(
    int t, bool live, int H, int E, int K, float eps, const XT* __restrict__ x,
    const float* __restrict__ pre_gain, const float* __restrict__ pes,
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const float* __restrict__ d_w, const float* __restrict__ d_logits, float (&dl)[4],
    float& beta, float (&dpes)[4]) {
  const int lane = lane_id();
#pragma unroll
  for (int j = 0; j < 4; ++j) dl[j] = 0.0f;
  beta = 0.0f;
  if (!live) return;  // uniform over the wave
  // in the order of what has to wait: the picks, x's row (3 pieces a lane at a
  // time: six took 104 registers and one block a CU, 8192 tokens 94 us in all
  // instead of 87), the logits, then what the picks point at
  int e = d_w != nullptr && lane < K ? topk_idx[(size_t)t * K + lane] : -1;
  const float dw = d_w != nullptr && lane < K ? d_w[(size_t)t * K + lane] : 0.0f;
  constexpr int XP = 3, XSTEP = 8 * kWave;
  const XT* xr = x + (size_t)t * H;
  Piece<XT> xp[XP];
  auto load_x = [&](int h0) {
#pragma unroll
    for (int i = 0; i < XP; ++i) xp[i].load(xr + min(h0 + i * XSTEP, H - 8));
  };
  load_x(8 * lane);
  float l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int ej = lane + kWave * j;
    l[j] = ej < E ? logits[(size_t)t * E + ej] : 0.0f;
    if (d_logits != nullptr && ej < E) dl[j] = d_logits[(size_t)t * E + ej];
    if (l[j] == -INFINITY) dl[j] = 0.0f;  // an expert switched off
  }
  // lane k < K: slot k (an id outside [0, E) or of an expert switched off is no slot)
  if ((unsigned)e >= (unsigned)E) e = -1;
  const float lk = e >= 0 ? logits[(size_t)t * E + e] : -INFINITY;
  const float pk = e >= 0 ? pes[e] : 0.0f;
  if (lk == -INFINITY) e = -1;
  float ss = 0.0f, sg = 0.0f;
  for (int h0 = 8 * lane;; h0 += XP * XSTEP) {
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int h = h0 + i * XSTEP;
      if (h >= H) break;
      float v[8];
      xp[i].get(v);
#pragma unroll
      for (int u = 0; u < 8; ++u) ss = __builtin_fmaf(v[u], v[u], ss);
      if (pre_gain != nullptr) {
        float g[8];
        load8f(pre_gain + h, g);
#pragma unroll
        for (int u = 0; u < 8; ++u) sg = __builtin_fmaf(v[u] * g[u], v[u] * g[u], sg);
      }
    }
    if (h0 - 8 * lane + XP * XSTEP >= H) break;  // uniform
    load_x(h0 + XP * XSTEP);
  }
  ss = group_sum<kWave>(ss);
  float r0 = 1.0f, r;
  if (pre_gain != nullptr) {
    sg = group_sum<kWave>(sg);
    r0 = 1.0f / sqrtf(ss / (float)H + eps);
    r = 1.0f / sqrtf(r0 * r0 * sg / (float)H + eps);
  } else {
    r = 1.0f / sqrtf(ss / (float)H + eps);
  }
  if (d_w != nullptr) {
    const float top = group_max<kWave>(lk);
    float q = lk == -INFINITY ? 0.0f : exp_neg(lk - top);
    const float z = group_sum<kWave>(q);
    q = z > 0.0f ? q / z : 0.0f;
    const float d = e >= 0 ? dw * pk : 0.0f;
    const float qd = group_sum<kWave>(q * d);
    const float dlk = q * (d - qd), dsk = e >= 0 ? dw * q : 0.0f;
    for (int k = 0; k < K; ++k) {  // a repeated id adds up
      const int ek = __builtin_amdgcn_readlane(e, k);
      const float dk = lane_value(dlk, k), sk = lane_value(dsk, k);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ek == lane + kWave * j) {
          dl[j] += dk;
          dpes[j] += sk;
        }
    }
  }
  float D = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) D += dl[j] != 0.0f ? dl[j] * l[j] : 0.0f;
  D = group_sum<kWave>(D);
  const float scale = r0 * r;
  beta = scale * scale * (D / (float)H);
#pragma unroll
  for (int j = 0; j < 4; ++j) dl[j] *= scale;
}

// The block's sums of dpes, added over its waves.
__device__ __forceinline__ void store_pes_part(float (*sums)[kMaxE], int waves, int E,
                                               const float (&dpes)[4], float* __restrict__ part) {
  const int wave = threadIdx.x / kWave, lane = lane_id();
#pragma unroll
  for (int j = 0; j < 4; ++j) sums[wave][lane + kWave * j] = dpes[j];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.0f;
    for (int w = 0; w < waves; ++w) s += sums[w][e];
    part[(size_t)blockIdx.x * E + e] = s;
  }
}

// fp32 inputs: dl' in fp32 [T, E].
__global__ __launch_bounds__(64 * kRgRowWaves) void router_grad_rows_kernel(
    int T, int H, int E, int K, float eps, const float* __restrict__ x,
    const float* __restrict__ pre_gain, const float* __restrict__ pes,
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const uint8_t* __restrict__ mask, const float* __restrict__ d_w,
    const float* __restrict__ d_logits, float* __restrict__ dl_out, float* __restrict__ beta_out,
    float* __restrict__ part_pes) {
  __shared__ float sums[kRgRowWaves][kMaxE];
  const int wave = threadIdx.x / kWave, lane = lane_id();
  float dpes[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // experts lane + 64 j
  for (int t = blockIdx.x * kRgRowWaves + wave; t < T; t += gridDim.x * kRgRowWaves) {
    float dl[4], beta;
    router_grad_token(t, mask == nullptr || mask[t] != 0, H, E, K, eps, x, pre_gain, pes, logits,
                      topk_idx, d_w, d_logits, dl, beta, dpes);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = lane + kWave * j;
      if (e < E) dl_out[(size_t)t * E + e] = dl[j];
    }
    if (lane == 0) beta_out[t] = beta;
  }
  store_pes_part(sums, kRgRowWaves, E, dpes, part_pes);
}

// fp32 matrix instruction 32x32x2: lane l holds A[l % 32][l / 32] and
// B[l / 32][l % 32]; register q of lane l is D[8 (q / 4) + 4 (l / 32) + q % 4]
// [l % 32].  One value of the contraction per lane and instruction: both
// operands come straight from rows whose fast axis is not the contraction.
__device__ __forceinline__ f32x16 mfma_f32(float a, float b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ int mfma_row(int q, int g) { return 8 * (q / 4) + 4 * g + q % 4; }

// G partial of one split of the tokens: a wave takes 32 MT experts x 64
// columns of x, the block's four waves four quarters of the split's tokens,
// added through LDS.  The wave also sums x^2 beta for its columns (experts'
// tile 0 only).  4096 tokens, 2816 x 128: 51 us (58 TF/s), the latency of loads that
// run one step ahead at two waves a SIMD; without that step and a wave a SIMD 81.
constexpr int kRgWaves = 4;
struct BlockAt { int col, y, z; };  // 64 columns; experts or tokens; split

// A launch of wb blocks that make G's partials and the rest dx, which need nothing
// of each other, spread evenly.  True for a block of G.
__device__ __forceinline__ bool grad_block(int wb, int H, int ey, BlockAt& at) {
  const long long n = gridDim.x, b = blockIdx.x, w = b * wb / n;
  const bool is_w = (b + 1) * wb / n != w;
  const int i = (int)(is_w ? w : b - w), cols = H / 64;
  at.col = i % cols;
  at.y = is_w ? i / cols % ey : i / cols;
  at.z = is_w ? i / cols / ey : 0;
  return is_w;
}

template <int MT>
__device__ __forceinline__ void router_grad_w(
    BlockAt at, int T, int H, int E, int span, const float* __restrict__ x,
    const uint8_t* __restrict__ mask, const float* __restrict__ dl,
    const float* __restrict__ beta, float* __restrict__ part_g, float* __restrict__ part_b) {
  __shared__ float acc_s[kRgWaves][16 * 2][kWave];
  __shared__ float b_s[kRgWaves][64];
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const int c = lane % 32, g = lane / 32;
  const int h0 = at.col * 64, e0 = at.y * 32 * MT, split = at.z;
  const int s0 = split * span, s1 = min(T, s0 + span);
  const int q4 = ((s1 - s0 + kRgWaves - 1) / kRgWaves + 1) / 2 * 2;
  const int t0 = min(s1, s0 + wave * q4), t1 = min(s1, t0 + q4);
  f32x16 acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  float bs[2] = {0.0f, 0.0f};
  // U pairs of tokens at a time, the next ones' loads on their way during a group's
  // products; a token past the last or a masked one counts as zeros, whatever its
  // rows hold
  constexpr int U = 2;
  float na[U][MT], nb[U][2], nbe[U];
  bool non[U];
  auto load = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tt = t + 2 * u + g, tc = min(tt, t1 - 1);
      non[u] = tt < t1 && (mask == nullptr || mask[tc] != 0);
#pragma unroll
      for (int i = 0; i < MT; ++i) na[u][i] = dl[(size_t)tc * E + min(e0 + 32 * i + c, E - 1)];
#pragma unroll
      for (int j = 0; j < 2; ++j) nb[u][j] = x[(size_t)tc * H + h0 + 32 * j + c];
      nbe[u] = beta[tc];
    }
  };
  if (t0 < t1) load(t0);
  for (int t = t0; t < t1; t += 2 * U) {
    float a[U][MT], b[U][2], be[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < MT; ++i) a[u][i] = non[u] && e0 + 32 * i + c < E ? na[u][i] : 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) b[u][j] = non[u] ? nb[u][j] : 0.0f;
      be[u] = non[u] ? nbe[u] : 0.0f;
    }
    load(min(t + 2 * U, t1 - 1));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma_f32(a[u][i], b[u][j], acc[i][j]);
#pragma unroll
      for (int j = 0; j < 2; ++j) bs[j] = __builtin_fmaf(b[u][j] * b[u][j], be[u], bs[j]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  const bool want_b = at.y == 0;
  if (want_b) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float v = bs[j] + __shfl_xor(bs[j], 32, kWave);
      if (g == 0) b_s[wave][32 * j + c] = v;
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc_s[wave][16 * j + q][lane] = acc[i][j][q];
    __syncthreads();
    // each wave adds a quarter of the 32 registers
#pragma unroll
    for (int k = 0; k < 32 / kRgWaves; ++k) {
      const int r = wave * (32 / kRgWaves) + k;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kRgWaves; ++w) v += acc_s[w][r][lane];
      const int e = e0 + 32 * i + mfma_row(r % 16, g), h = h0 + 32 * (r / 16) + c;
      if (e < E) part_g[((size_t)split * E + e) * H + h] = v;
    }
  }
  if (want_b && threadIdx.x < 64) {
    float v = 0.0f;
    for (int w = 0; w < kRgWaves; ++w) v += b_s[w][threadIdx.x];
    part_b[(size_t)split * H + h0 + threadIdx.x] = v;
  }
}

// dx: a wave takes 64 tokens x 64 columns; the contraction runs over the
// experts, four per lane and load (lanes 0-31 experts 8 s .. 8 s + 3, lanes
// 32-63 the next four; W's rows in the same order).  4096 tokens, 2816 x 128: 82 us
// (36 TF/s), 32 lines of dl' and 8 of W a step of 16 products; with no step ahead and
// the tokens' factors loaded again for every 32 columns 123.
__device__ __forceinline__ void router_grad_x(
    BlockAt at, bool vec, int T, int H, int E, float eps, const float* __restrict__ x,
    const uint8_t* __restrict__ mask,
    const float* __restrict__ dl, const float* __restrict__ beta, const float* __restrict__ W,
    const float* __restrict__ scale, const float* __restrict__ pre_gain, float* __restrict__ dx) {
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const int c = lane % 32, g = lane / 32;
  const int h0 = at.col * 64, t0 = (at.y * kRgWaves + wave) * 64;
  if (t0 >= T) return;  // no barrier below
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  float na[2][4], nb[4][2];  // of the next step
  auto load = [&](int e0) __attribute__((always_inline)) {
    const int e = e0 + 4 * g;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* row = dl + (size_t)min(t0 + 32 * i + c, T - 1) * E;
      if (vec) {  // E % 4 == 0: all four exist or none
        const float4 v = *reinterpret_cast<const float4*>(row + min(e, E - 4));
        na[i][0] = v.x; na[i][1] = v.y; na[i][2] = v.z; na[i][3] = v.w;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) na[i][k] = row[min(e + k, E - 1)];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) nb[k][j] = W[(size_t)min(e + k, E - 1) * H + h0 + 32 * j + c];
  };
  load(0);
  for (int e0 = 0; e0 < E; e0 += 8) {
    float a[2][4], b[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool on = e0 + 4 * g + k < E;
#pragma unroll
      for (int i = 0; i < 2; ++i) a[i][k] = on ? na[i][k] : 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) b[k][j] = on ? nb[k][j] : 0.0f;
    }
    load(min(e0 + 8, E - 1));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma_f32(a[i][k], b[k][j], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
  }
  float gc[2], ge[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int h = h0 + 32 * j + c;
    const float gn = pre_gain != nullptr ? pre_gain[h] : 1.0f;
    gc[j] = gn * scale[h];
    ge[j] = pre_gain != nullptr ? gn * gn + eps : 1.0f;
  }
  // 32 tokens' loads all before their first store
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float xv[2][16], be[16];
    bool on[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int t = min(t0 + 32 * i + mfma_row(q, g), T - 1);
      on[q] = mask == nullptr || mask[t] != 0;
      be[q] = beta[t];
#pragma unroll
      for (int j = 0; j < 2; ++j) xv[j][q] = x[(size_t)t * H + h0 + 32 * j + c];
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int t = t0 + 32 * i + mfma_row(q, g);
      if (t < T)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          dx[(size_t)t * H + h0 + 32 * j + c] =
              on[q] ? gc[j] * acc[i][j][q] - xv[j][q] * (be[q] * ge[j]) : 0.0f;
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int MT>
__global__ __launch_bounds__(64 * kRgWaves, 2) void router_grad_wx_kernel(
    int wb, int ey, int T, int H, int E, int span, float eps, const float* __restrict__ x,
    const uint8_t* __restrict__ mask, const float* __restrict__ dl,
    const float* __restrict__ beta, const float* __restrict__ W, const float* __restrict__ scale,
    const float* __restrict__ pre_gain, float* __restrict__ part_g, float* __restrict__ part_b,
    float* __restrict__ dx) {
  BlockAt at;
  if (grad_block(wb, H, ey, at))
    router_grad_w<MT>(at, T, H, E, span, x, mask, dl, beta, part_g, part_b);
  else
    router_grad_x(at, E % 4 == 0, T, H, E, eps, x, mask, dl, beta, W, scale, pre_gain, dx);
}

__global__ __launch_bounds__(64 * kRgWaves, 2) void router_grad_x_kernel(
    int T, int H, int E, float eps, const float* __restrict__ x, const uint8_t* __restrict__ mask,
    const float* __restrict__ dl, const float* __restrict__ beta, const float* __restrict__ W,
    const float* __restrict__ scale, const float* __restrict__ pre_gain, float* __restrict__ dx) {
  BlockAt at;
  grad_block(0, H, 1, at);
  router_grad_x(at, E % 4 == 0, T, H, E, eps, x, mask, dl, beta, W, scale, pre_gain, dx);
}

// ---------------------------------------------------------------------------
// bf16 inputs: both products on bf16 matrix instructions (16x16x32: lane l holds
// row l % 16 of each operand, k = 8 (l / 16) .. + 7; register r of the result
// is row 4 (l / 16) + r of the first operand, row l % 16 of the second).  x is
// bf16 already; dl' and W are cut into bf16 parts, v = v0 + v1 + v2 with v0 the
// value rounded and v1, v2 the rest rounded: three parts hold all 24 bits, two
// hold 16.  G = dl'^T x takes the three parts (an fp32 result); dx, rounded to
// bf16 at the end, the products v0 w0 + v0 w1 + v1 w0, which leave out 2^-16.
// A third of the fp32 instruction's time and less (it takes 16 times as long
// for the same product).
//
// The rows kernel stores every operand in the order in which a wave loads it, a
// fragment of 64 lanes x 16 bytes at a time (row-major parts, whose loads touch
// 64 bytes of 16 rows, took the products 28 of 42 us at 4096 tokens).  Ep and Tp:
// experts and tokens rounded up to 32, zeros past the end.
//   dl' for dx  [Tp / 16][Ep / 32][2 parts][lane]   token 16 i + l % 16, experts
//                                                   32 k + 8 (l / 16) .. + 7
//   dl' for G   [Tp / 32][Ep / 16][3 parts][lane]   expert 16 m + l % 16, tokens
//                                                   32 s + 8 (l / 16) .. + 7
//   W for dx    [H / 16][Ep / 32][2 parts][lane]    column wt_col(l % 16) of the
//                                                   tile, experts as in dl'
// ---------------------------------------------------------------------------
constexpr int kRgSumBytes = 2 * kRgWaves * 4 * kWave * 16;  // two tiles' results per wave
constexpr int kRgTok = 16;   // tokens per rows block, one per wave
constexpr int kRgRowThreads = kRgTok * kWave;
constexpr int kRgWCols = 32; // columns of W per block past those

constexpr int kFrag = kWave * 8;  // values of a fragment

// Column of row m of the 16-column tile i of W^T, counted from the first of the
// 32 columns of tiles i and i + 1 (i even): a lane's results of the two tiles
// (rows 4 g .. 4 g + 3 of each) are then eight consecutive columns.
__device__ __forceinline__ int wt_col(int i, int m) { return 8 * (m / 4) + 4 * (i % 2) + m % 4; }

__device__ __forceinline__ void split3(float v, bf16& a, bf16& b, bf16& c) {
  a = (bf16)v;
  const float r = v - (float)a;
  b = (bf16)r;
  c = (bf16)(r - (float)b);
}

__global__ __launch_bounds__(kRgRowThreads, 8) void router_grad_rows_bf16_kernel(
    int T, int H, int E, int K, float eps, const bf16* __restrict__ x,
    const float* __restrict__ pre_gain, const float* __restrict__ pes,
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const uint8_t* __restrict__ mask, const float* __restrict__ d_w,
    const float* __restrict__ d_logits, const float* __restrict__ W, int tok_blocks,
    bf16* __restrict__ rows_out, bf16* __restrict__ cols_out, bf16* __restrict__ wt_out,
    float* __restrict__ beta_out, uint8_t* __restrict__ live_out, float* __restrict__ part_pes) {
  __shared__ float tile[kRgWCols][kMaxE + 1];  // W^T's columns, or kRgTok tokens' dl'
  __shared__ float sums[kRgTok][kMaxE];
  const int tid = threadIdx.x, wave = tid / kWave, lane = lane_id();
  const int Ep = (E + 31) / 32 * 32;
  if ((int)blockIdx.x >= tok_blocks) {  // columns of W, transposed
    const int h0 = ((int)blockIdx.x - tok_blocks) * kRgWCols;
    const int c = tid % kRgWCols;
#pragma unroll 8
    for (int e = tid / kRgWCols; e < Ep; e += kRgRowThreads / kRgWCols)
      tile[c][e] = e < E ? W[(size_t)e * H + h0 + c] : 0.0f;
    __syncthreads();
    const int KS = Ep / 32;
    // tiles h0 / 16 and h0 / 16 + 1
    for (int k = tid; k < 2 * KS * kWave; k += kRgRowThreads) {
      const int l = k % kWave, ks = k / kWave % KS, i = k / kWave / KS;
      const int col = wt_col(i, l % 16), e0 = 32 * ks + 8 * (l / 16);
      bf16x8 p[2];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        bf16 a, b, c;
        split3(tile[col][e0 + u], a, b, c);
        p[0][u] = a;
        p[1][u] = b;
      }
      bf16* dst = wt_out + ((size_t)(h0 / 16 + i) * KS + ks) * 2 * kFrag + 8 * l;
      *reinterpret_cast<bf16x8*>(dst) = p[0];
      *reinterpret_cast<bf16x8*>(dst + kFrag) = p[1];
    }
    return;
  }
  const int t0 = blockIdx.x * kRgTok;
  float dpes[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  {
    const int t = t0 + wave;
    const bool live = t < T && (mask == nullptr || mask[t] != 0);
    float dl[4], beta;
    router_grad_token(t, live, H, E, K, eps, x, pre_gain, pes, logits, topk_idx, d_w, d_logits,
                      dl, beta, dpes);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + kWave * j < Ep) tile[wave][lane + kWave * j] = dl[j];
    if (lane == 0) {  // [Tp]: zeros past the last token
      beta_out[t] = beta;
      live_out[t] = live ? 1 : 0;
    }
  }
  store_pes_part(sums, kRgTok, E, dpes, part_pes);  // (its barrier covers the tile)
  const int KS = Ep / 32, MS = Ep / 16;
  for (int k = tid; k < KS * kWave; k += kRgRowThreads) {
    const int l = k % kWave, ks = k / kWave, tl = l % 16, e0 = 32 * ks + 8 * (l / 16);
    bf16x8 p[2];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      bf16 a, b, c;
      split3(tile[tl][e0 + u], a, b, c);
      p[0][u] = a;
      p[1][u] = b;
    }
    bf16* dst = rows_out + ((size_t)blockIdx.x * KS + ks) * 2 * kFrag + 8 * l;
    *reinterpret_cast<bf16x8*>(dst) = p[0];
    *reinterpret_cast<bf16x8*>(dst + kFrag) = p[1];
  }
  // the block's 16 tokens are half a step: lane groups 0, 1 or 2, 3
  for (int k = tid; k < MS * 32; k += kRgRowThreads) {
    const int l = k % 32, m = k / 32, e = 16 * m + l % 16, tl = 8 * (l / 16);
    bf16x8 p[3];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      bf16 a, b, c;
      split3(tile[tl + u][e], a, b, c);
      p[0][u] = a;
      p[1][u] = b;
      p[2][u] = c;
    }
    bf16* dst = cols_out + ((size_t)(blockIdx.x / 2) * MS + m) * 3 * kFrag +
                8 * (l + 32 * (blockIdx.x % 2));
#pragma unroll
    for (int q = 0; q < 3; ++q) *reinterpret_cast<bf16x8*>(dst + q * kFrag) = p[q];
  }
}

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// G partial: a wave takes 16 MT experts x 64 columns of x over a quarter of the
// split's 32-token steps.  x rows are loaded as they lie, four columns of eight
// tokens a lane, and regrouped in registers: fragment i holds columns 4 (l % 16)
// + i, so a lane's four results of a row are consecutive columns.  The next
// step's x and parts of dl' are fetched during a step's products; what is left
// is their latency (19.8 us at 4096 tokens of 2816, 128 experts; two column groups
// a block, which halves what L2 delivers, took as long).
template <int MT, bool MASK>
__device__ __forceinline__ void router_grad_w_bf16(
    BlockAt at, unsigned char* smem, int T, int H, int E, int steps, const bf16* __restrict__ x,
    const uint8_t* __restrict__ live,
    const bf16* __restrict__ cols, const float* __restrict__ beta, bool want_beta,
    float* __restrict__ part_g, float* __restrict__ part_b) {
  auto acc_s = reinterpret_cast<f32x4 (*)[kRgWaves][4][kWave]>(smem);  // [2]
  auto b_s = reinterpret_cast<float (*)[4][64]>(smem + kRgSumBytes);   // [kRgWaves]
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const int c = lane % 16, g = lane / 16;
  const int h0 = at.col * 64, m0 = at.y * MT, split = at.z;
  const int MS = (E + 31) / 32 * 2, all = (T + 31) / 32;
  const int s0 = min(all, split * steps), s1 = min(all, s0 + steps);
  const int n = s1 - s0, a0 = s0 + wave * n / kRgWaves, a1 = s0 + (wave + 1) * n / kRgWaves;
  const bool beta_here = want_beta && at.y == 0;
  f32x4 acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = f32x4{0, 0, 0, 0};
  float bs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  uint2 raw[8], on = {0u, 0u};
  float4 be4[2] = {};
  // (steps past the wave's last load that one again)
  auto load_x = [&](int s) {
    if constexpr (MASK) on = *reinterpret_cast<const uint2*>(live + 32 * s + 8 * g);
    if (beta_here) {
      be4[0] = *reinterpret_cast<const float4*>(beta + 32 * s + 8 * g);
      be4[1] = *reinterpret_cast<const float4*>(beta + 32 * s + 8 * g + 4);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = min(32 * s + 8 * g + j, T - 1);
      raw[j] = *reinterpret_cast<const uint2*>(x + (size_t)t * H + h0 + 4 * c);
    }
  };
  bf16x8 fa[2][MT][3];
  auto load_a = [&](int s, bf16x8 (&f)[MT][3]) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const bf16* p = cols + ((size_t)s * MS + min(m0 + m, MS - 1)) * 3 * kFrag + 8 * lane;
#pragma unroll
      for (int q = 0; q < 3; ++q) f[m][q] = *reinterpret_cast<const bf16x8*>(p + q * kFrag);
    }
  };
  if (a0 < a1) {
    load_x(a0);
    load_a(a0, fa[0]);
  }
  // one step, its parts in fa[cur]; the next step's x and parts are on their way
  // during its products
  auto step = [&](int s, auto cur_tag) __attribute__((always_inline)) {
    constexpr int now = decltype(cur_tag)::value;
    const int next = min(s + 1, a1 - 1);
    uint2 cur[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cur[j] = raw[j];
      if constexpr (MASK) {  // a masked row may hold anything
        const uint32_t w = j < 4 ? on.x : on.y;
        if (((w >> (8 * (j % 4))) & 255u) == 0) cur[j] = make_uint2(0u, 0u);
      }
    }
    const float4 b0 = be4[0], b1 = be4[1];
    load_x(next);
    load_a(next, fa[1 - now]);
    __builtin_amdgcn_sched_barrier(0);
    if (beta_here) {
      const float bb[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float be = bb[j];
        const float v[4] = {__uint_as_float(cur[j].x << 16),
                            __uint_as_float(cur[j].x & 0xffff0000u),
                            __uint_as_float(cur[j].y << 16),
                            __uint_as_float(cur[j].y & 0xffff0000u)};
#pragma unroll
        for (int i = 0; i < 4; ++i) bs[i] = __builtin_fmaf(v[i] * v[i], be, bs[i]);
      }
    }
    // columns 4 c + i of the eight tokens: halves of eight words
    bf16x8 fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 w;
      uint32_t* wp = &w.x;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t lo = i < 2 ? cur[2 * p].x : cur[2 * p].y;
        const uint32_t hi = i < 2 ? cur[2 * p + 1].x : cur[2 * p + 1].y;
        wp[p] = i % 2 == 0 ? __builtin_amdgcn_perm(hi, lo, 0x05040100u)
                           : __builtin_amdgcn_perm(hi, lo, 0x07060302u);
      }
      fb[i] = __builtin_bit_cast(bf16x8, w);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = mfma_bf16(fa[now][m][q], fb[i], acc[m][i]);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int s = a0; s < a1; s += 2) {
    step(s, std::integral_constant<int, 0>{});
    if (s + 1 < a1) step(s + 1, std::integral_constant<int, 1>{});
  }
  if (beta_here) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b_s[wave][g][4 * c + i] = bs[i];
  }
#pragma unroll
  for (int m = 0; m < MT; m += 2) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc_s[d][wave][i][lane] = acc[m + d][i];
    __syncthreads();
    // wave w adds result register w of every lane: row 4 g + w, columns 4 c .. + 3
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = 0.0f;
#pragma unroll
        for (int u = 0; u < kRgWaves; ++u) v[i] += acc_s[d][u][i][lane][wave];
      }
      const int e = 16 * (m0 + m + d) + 4 * g + wave;
      if (e < E)
        *reinterpret_cast<f32x4*>(part_g + ((size_t)split * E + e) * H + h0 + 4 * c) = v;
    }
  }
  if (beta_here && threadIdx.x < 64) {
    float v = 0.0f;
    for (int w = 0; w < kRgWaves; ++w)
      for (int i = 0; i < 4; ++i) v += b_s[w][i][threadIdx.x];
    part_b[(size_t)split * H + h0 + threadIdx.x] = v;
  }
}

// dx: a block takes 64 columns x 32 WAVES tokens, a wave 32 of the tokens.  The columns'
// W^T fragments go to LDS once (32 KB at 128 experts), the tokens' fragments and
// the rows of x come straight from memory, one step ahead.  W^T is the first
// operand: with its column order (wt_col) a lane's results of two tiles are eight
// consecutive columns of a token, 16-byte loads of x and stores of dx.
constexpr int kRgXTok = 32;
template <int WAVES>
__device__ __forceinline__ void router_grad_x_bf16(
    BlockAt at, unsigned char* smem, int T, int H, int E, float eps, const bf16* __restrict__ x,
    const uint8_t* __restrict__ live,
    const bf16* __restrict__ rows, const float* __restrict__ beta, const bf16* __restrict__ wt,
    const float* __restrict__ scale, const float* __restrict__ pre_gain, bf16* __restrict__ dx) {
  bf16x8* ws = reinterpret_cast<bf16x8*>(smem);  // [4 tiles][KS][2][lane]
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane % 16, g = lane / 16;
  const int h0 = at.col * 64, t0 = (at.y * WAVES + wave) * kRgXTok;
  const int KS = (E + 31) / 32, tiles = (T + 31) / 32 * 2;
  const bf16* tr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    tr[i] = rows + (size_t)min(t0 / 16 + i, tiles - 1) * KS * 2 * kFrag + 8 * lane;
  bf16x8 ft[2][2];  // [token tile][part]
  auto load_t = [&](int k) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        ft[i][q] = *reinterpret_cast<const bf16x8*>(tr[i] + (2 * k + q) * kFrag);
  };
  load_t(0);
  Piece<bf16> xp[2][2];  // [token tile][column pair]
  float be[2];
  bool on[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = min(t0 + 16 * i + c, T - 1);
    be[i] = beta[t];
    on[i] = live[t] != 0;
#pragma unroll
    for (int p = 0; p < 2; ++p) xp[i][p].load(x + (size_t)t * H + h0 + 32 * p + 8 * g);
  }
  const bf16x8* src = reinterpret_cast<const bf16x8*>(wt + (size_t)h0 / 16 * KS * 2 * kFrag);
#pragma unroll 4
  for (int k = tid; k < 4 * KS * 2 * kWave; k += 64 * WAVES) ws[k] = src[k];
  __syncthreads();
  f32x4 acc[2][4];  // token tile, column tile
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  for (int k = 0; k < KS; ++k) {
    bf16x8 cur[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) cur[i][q] = ft[i][q];
    load_t(min(k + 1, KS - 1));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 w0 = ws[((j * KS + k) * 2) * kWave + lane];
      const bf16x8 w1 = ws[((j * KS + k) * 2 + 1) * kWave + lane];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        acc[i][j] = mfma_bf16(w0, cur[i][1], acc[i][j]);
        acc[i][j] = mfma_bf16(w1, cur[i][0], acc[i][j]);
        acc[i][j] = mfma_bf16(w0, cur[i][0], acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {  // columns h .. h + 7
    const int h = h0 + 32 * p + 8 * g;
    float gc[8], gn[8], ge[8];
    load8f(scale + h, gc);
    if (pre_gain != nullptr) load8f(pre_gain + h, gn);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      ge[u] = pre_gain != nullptr ? gn[u] * gn[u] + eps : 1.0f;
      if (pre_gain != nullptr) gc[u] *= gn[u];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + 16 * i + c;
      if (t >= T) continue;
      float xv[8];
      xp[i][p].get(xv);
      bf16x8 o;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float v = gc[u] * acc[i][2 * p + u / 4][u % 4] - xv[u] * (be[i] * ge[u]);
        o[u] = (bf16)(on[i] ? v : 0.0f);
      }
      *reinterpret_cast<bf16x8*>(dx + (size_t)t * H + h) = o;
    }
  }
}

constexpr int kRgWBytes = kRgSumBytes + kRgWaves * 4 * 64 * 4;
template <int MT, bool MASK>
__global__ __launch_bounds__(64 * kRgWaves, 2) void router_grad_wx_bf16_kernel(
    int wb, int ey, int T, int H, int E, int steps, float eps, const bf16* __restrict__ x,
    const uint8_t* __restrict__ live, const bf16* __restrict__ rows,
    const bf16* __restrict__ cols, const float* __restrict__ beta, const bf16* __restrict__ wt,
    const float* __restrict__ scale, const float* __restrict__ pre_gain,
    float* __restrict__ part_g, float* __restrict__ part_b, bf16* __restrict__ dx) {
  extern __shared__ __align__(16) unsigned char smem[];
  BlockAt at;
  if (grad_block(wb, H, ey, at))
    router_grad_w_bf16<MT, MASK>(at, smem, T, H, E, steps, x, live, cols, beta,
                                 pre_gain != nullptr, part_g, part_b);
  else
    router_grad_x_bf16<kRgWaves>(at, smem, T, H, E, eps, x, live, rows, beta, wt, scale, pre_gain,
                                 dx);
}

constexpr int kRgXWaves = 8;
__global__ __launch_bounds__(64 * kRgXWaves, 4) void router_grad_x_bf16_kernel(
    int T, int H, int E, float eps, const bf16* __restrict__ x, const uint8_t* __restrict__ live,
    const bf16* __restrict__ rows, const float* __restrict__ beta, const bf16* __restrict__ wt,
    const float* __restrict__ scale, const float* __restrict__ pre_gain, bf16* __restrict__ dx) {
  extern __shared__ __align__(16) unsigned char smem[];
  router_grad_x_bf16<kRgXWaves>(BlockAt{(int)blockIdx.x, (int)blockIdx.y, 0}, smem, T, H, E, eps,
                                x, live, rows, beta, wt, scale, pre_gain, dx);
}

// dx for many tokens, up to 128 experts: a block keeps the W^T of its 64 columns in
// LDS and its waves go through tiles of 16 tokens, the next tile's fragments, all of
// them, and rows of x on their way during a tile's products.  As many blocks as one
// round holds.  The whole backward of 4096 / 8192 tokens, 2816 x 128, 58.1 / 92.3 us
// with the kernel above, 55.1 / 81.9 with this one (and 3 pieces of x a lane in the
// first kernel); 256 experts, whose fragments take twice the registers, 79.6 and
// 81.7 at 4096 tokens.
constexpr int kRgXSteps = 4;  // of 32 experts, at most
__global__ __launch_bounds__(64 * kRgXWaves, 4) void router_grad_x_loop_kernel(
    int T, int H, int E, int span, float eps, const bf16* __restrict__ x,
    const uint8_t* __restrict__ live, const bf16* __restrict__ rows,
    const float* __restrict__ beta, const bf16* __restrict__ wt,
    const float* __restrict__ scale, const float* __restrict__ pre_gain, bf16* __restrict__ dx) {
  extern __shared__ __align__(16) unsigned char smem[];
  bf16x8* ws = reinterpret_cast<bf16x8*>(smem);  // [4 tiles][KS][2][lane]
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane % 16, g = lane / 16, h0 = blockIdx.x * 64;
  const int KS = (E + 31) / 32, tiles = (T + 15) / 16;
  const int i0 = blockIdx.y * span, i1 = min(tiles, i0 + span);
  bf16x8 ft[kRgXSteps][2];
  Piece<bf16> xp[2];
  float be = 0.0f;
  bool on = false;
  auto load = [&](int i) __attribute__((always_inline)) {
    const bf16* p = rows + (size_t)i * KS * 2 * kFrag + 8 * lane;
#pragma unroll
    for (int k = 0; k < kRgXSteps; ++k)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        ft[k][q] = *reinterpret_cast<const bf16x8*>(p + (2 * min(k, KS - 1) + q) * kFrag);
    const int t = min(16 * i + c, T - 1);
#pragma unroll
    for (int p2 = 0; p2 < 2; ++p2) xp[p2].load(x + (size_t)t * H + h0 + 32 * p2 + 8 * g);
    be = beta[t];
    on = live[t] != 0;
  };
  int i = i0 + wave;
  if (i < i1) load(i);
  const bf16x8* src = reinterpret_cast<const bf16x8*>(wt + (size_t)h0 / 16 * KS * 2 * kFrag);
#pragma unroll 4
  for (int k = tid; k < 4 * KS * 2 * kWave; k += 64 * kRgXWaves) ws[k] = src[k];
  // [2][64]: the columns' factors
  float* gs = reinterpret_cast<float*>(smem + 64 * kRgXSteps * 32 * 4);
  if (tid < 64) {
    const float gn = pre_gain != nullptr ? pre_gain[h0 + tid] : 1.0f;
    gs[tid] = gn * scale[h0 + tid];
    gs[64 + tid] = pre_gain != nullptr ? gn * gn + eps : 1.0f;
  }
  __syncthreads();
  for (; i < i1; i += kRgXWaves) {
    bf16x8 f[kRgXSteps][2];
#pragma unroll
    for (int k = 0; k < kRgXSteps; ++k)
#pragma unroll
      for (int q = 0; q < 2; ++q) f[k][q] = ft[k][q];
    const Piece<bf16> x0 = xp[0], x1 = xp[1];
    const float b = be;
    const bool live_t = on;
    const int t = 16 * i + c;
    if (i + kRgXWaves < i1) load(i + kRgXWaves);
    f32x4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kRgXSteps; ++k) {
      if (k >= KS) break;  // uniform
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 w0 = ws[((j * KS + k) * 2) * kWave + lane];
        const bf16x8 w1 = ws[((j * KS + k) * 2 + 1) * kWave + lane];
        acc[j] = mfma_bf16(w0, f[k][1], acc[j]);
        acc[j] = mfma_bf16(w1, f[k][0], acc[j]);
        acc[j] = mfma_bf16(w0, f[k][0], acc[j]);
      }
    }
    if (t >= T) continue;
#pragma unroll
    for (int p = 0; p < 2; ++p) {  // columns h0 + 32 p + 8 g .. + 7
      float xv[8], gc[8], ge[8];
      (p == 0 ? x0 : x1).get(xv);
      load8f(gs + 32 * p + 8 * g, gc);
      load8f(gs + 64 + 32 * p + 8 * g, ge);
      bf16x8 o;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float v = gc[u] * acc[2 * p + u / 4][u % 4] - xv[u] * (b * ge[u]);
        o[u] = (bf16)(live_t ? v : 0.0f);
      }
      *reinterpret_cast<bf16x8*>(dx + (size_t)t * H + h0 + 32 * p + 8 * g) = o;
    }
  }
}

// Last kernel: adds the splits of G; dW, dc and dg of 32 columns per block, four
// columns a thread and 32 groups of experts; in the blocks past the columns the
// per-expert scale's gradient from the first kernel's sums.  Its few blocks wait for
// memory: all the loads of a thread's EU experts go out before the first is added
// (128 experts, 2816 columns, 5 splits: 7.4 -> 5.5 us).
constexpr int kRgCols = 32, kRgParts = 32;  // thread rows, as many as splits or more
constexpr int kRgFinThreads = kRgCols / 4 * kRgParts;
template <int EU>
__global__ __launch_bounds__(kRgFinThreads) void router_grad_finish_kernel(
    int H, int E, int splits, int pes_blocks, const float* __restrict__ part_g,
    const float* __restrict__ part_b, const float* __restrict__ part_pes,
    const float* __restrict__ W, const float* __restrict__ scale,
    const float* __restrict__ pre_gain, float* __restrict__ dW, float* __restrict__ d_scale,
    float* __restrict__ d_pes, float* __restrict__ d_gain) {
  __shared__ f32x4 red[kRgParts][kRgCols / 4], red_b[kRgParts][kRgCols / 4];
  const int c = threadIdx.x % (kRgCols / 4), p = threadIdx.x / (kRgCols / 4);
  const int col_blocks = H / kRgCols;
  if ((int)blockIdx.x >= col_blocks) {
    // eight experts a block
    const int e = ((int)blockIdx.x - col_blocks) * (kRgCols / 4) + c;
    float s = 0.0f;
    if (e < E) {
#pragma unroll 8
      for (int i = p; i < pes_blocks; i += kRgParts) s += part_pes[(size_t)i * E + e];
    }
    red[p][c][0] = s;
    __syncthreads();
    if (p == 0 && e < E) {
      s = 0.0f;
      for (int i = 0; i < kRgParts; ++i) s += red[i][c][0];
      d_pes[e] = s;
    }
    return;
  }
  const int h = blockIdx.x * kRgCols + 4 * c;
  const f32x4 one = {1.0f, 1.0f, 1.0f, 1.0f};
  const f32x4 gn = pre_gain != nullptr ? *reinterpret_cast<const f32x4*>(pre_gain + h) : one;
  const f32x4 cs = *reinterpret_cast<const f32x4*>(scale + h);
  f32x4 m = {0.0f, 0.0f, 0.0f, 0.0f};
  // thread row p adds split p's sum of x^2 beta (at most kRgParts splits)
  f32x4 bsum = m;
  if (d_gain != nullptr && p < splits)
    bsum = *reinterpret_cast<const f32x4*>(part_b + (size_t)p * H + h);
  constexpr int U = 5;  // splits loaded before the first is added
  for (int e0 = p; e0 < E; e0 += EU * kRgParts) {
    f32x4 sum[EU], w[EU];
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      sum[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      w[i] = *reinterpret_cast<const f32x4*>(W + (size_t)min(e0 + i * kRgParts, E - 1) * H + h);
    }
    for (int s0 = 0; s0 < splits; s0 += U) {
      f32x4 v[EU][U];
#pragma unroll
      for (int i = 0; i < EU; ++i)
#pragma unroll
        for (int u = 0; u < U; ++u)
          v[i][u] = *reinterpret_cast<const f32x4*>(
              part_g +
              ((size_t)min(s0 + u, splits - 1) * E + min(e0 + i * kRgParts, E - 1)) * H + h);
#pragma unroll
      for (int i = 0; i < EU; ++i)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (s0 + u < splits) sum[i] += v[i][u];
    }
#pragma unroll
    for (int i = 0; i < EU; ++i) {
      const int e = e0 + i * kRgParts;
      if (e >= E) break;
      *reinterpret_cast<f32x4*>(dW + (size_t)e * H + h) = sum[i] * gn * cs;
      m += w[i] * sum[i];
    }
  }
  red[p][c] = m;
  red_b[p][c] = bsum;
  __syncthreads();
  if (p != 0) return;
  m = red[0][c];
#pragma unroll 8
  for (int i = 1; i < kRgParts; ++i) m += red[i][c];
  *reinterpret_cast<f32x4*>(d_scale + h) = gn * m;
  if (d_gain != nullptr) {
    for (int i = 1; i < splits; ++i) bsum += red_b[i][c];
    *reinterpret_cast<f32x4*>(d_gain + h) = cs * m - gn * bsum;
  }
}

// G's partials and dx take one launch where dx and a split of G (fp32, whose G takes
// longer: two) fit into one round of blocks, two a CU with bf16 inputs, one with
// fp32.  At 26B-A4B's shape, all of the router's backward: bf16 48 / 301 / 1024
// tokens 22.6 / 28.9 / 34.2 us in two launches, 19.0 / 24.4 / 31.0 in one (2048, forced:
// 43.5 in both); fp32 48 / 301 / 768 tokens 39.3 / 56.7 / 66.9 and 30.1 / 45.8 / 48.9
// (1024, forced: 70.6 and 93.6).
constexpr int kRgRound = 512;
int grad_round(bool bf16_in) { return bf16_in ? kRgRound : kRgRound / 2; }
int grad_w_blocks(int H, int E, bool bf16_in) {  // of a split
  const int experts = bf16_in ? 64 : 128;        // of a block
  return H / 64 * ((E + experts - 1) / experts);
}
// Splits of the tokens for G: one per 64 tokens, as many as two blocks a CU take in
// one round (26B-A4B's shape: bf16 5, fp32 11), 32 at most; beside dx in one launch
// what dx leaves of a round.
int grad_max_splits(int T, int H, int E, bool bf16_in) {
  const int by_cus = kRgRound / grad_w_blocks(H, E, bf16_in), by_tokens = (T + 63) / 64;
  const int n = by_cus < by_tokens ? by_cus : by_tokens;
  return n < 1 ? 1 : n < 32 ? n : 32;
}
int grad_x_blocks(int T, int H, bool bf16_in) {
  const int tok = kRgWaves * (bf16_in ? kRgXTok : 64);
  return H / 64 * ((T + tok - 1) / tok);
}
bool grad_one_launch(int T, int H, int E, bool bf16_in) {
  return grad_x_blocks(T, H, bf16_in) + grad_w_blocks(H, E, bf16_in) * (bf16_in ? 1 : 2) <=
         grad_round(bf16_in);
}
int grad_splits(int T, int H, int E, bool bf16_in) {
  const int most = grad_max_splits(T, H, E, bf16_in);
  if (!grad_one_launch(T, H, E, bf16_in)) return most;
  const int n = (grad_round(bf16_in) - grad_x_blocks(T, H, bf16_in)) /
                grad_w_blocks(H, E, bf16_in);
  return n < 1 ? 1 : n < most ? n : most;
}

// fp32 inputs.
void launch_grad_f32(const RouterGradArgs& a, hipStream_t s) {
  const float* x = static_cast<const float*>(a.x);
  float* dl = static_cast<float*>(a.ws_dl);
  const int splits = grad_splits(a.T, a.H, a.E, false);
  const bool one = a.d_x != nullptr && grad_one_launch(a.T, a.H, a.E, false);
  hipLaunchKernelGGL(router_grad_rows_kernel, dim3(router_grad_row_blocks(a.T)),
                     dim3(64 * kRgRowWaves), 0, s, a.T, a.H, a.E, a.K, a.eps, x, a.pre_gain,
                     a.per_expert_scale, a.logits, a.topk_idx, a.mask, a.d_topk_w, a.d_logits, dl,
                     a.ws_beta, a.ws_part_pes);
  const int span = (a.T + splits - 1) / splits;
  auto gw = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    const int cols = a.H / 64, ey = (a.E + 32 * MT - 1) / (32 * MT), wb = cols * ey * splits;
    const int xb = one ? grad_x_blocks(a.T, a.H, false) : 0;
    hipLaunchKernelGGL((router_grad_wx_kernel<MT>), dim3(wb + xb), dim3(64 * kRgWaves), 0, s, wb,
                       ey, a.T, a.H, a.E, span, a.eps, x, a.mask, dl, a.ws_beta, a.router_w,
                       a.router_scale, a.pre_gain, a.ws_part_g, a.ws_part_b,
                       static_cast<float*>(a.d_x));
  };
  if (a.E <= 32) gw(std::integral_constant<int, 1>{});
  else if (a.E <= 64) gw(std::integral_constant<int, 2>{});
  else gw(std::integral_constant<int, 4>{});
  if (a.d_x != nullptr && !one)
    hipLaunchKernelGGL(router_grad_x_kernel, dim3(grad_x_blocks(a.T, a.H, false)),
                       dim3(64 * kRgWaves), 0, s, a.T, a.H, a.E, a.eps, x, a.mask, dl, a.ws_beta,
                       a.router_w, a.router_scale, a.pre_gain, static_cast<float*>(a.d_x));
}

// bf16 inputs.
void launch_grad_bf16(const RouterGradArgs& a, hipStream_t s) {
  const bf16* x = static_cast<const bf16*>(a.x);
  const long long Ep = (a.E + 31) / 32 * 32, Tp = (a.T + 31) / 32 * 32;
  bf16* rows = static_cast<bf16*>(a.ws_dl);
  bf16* cols = rows + 2 * Tp * Ep;
  bf16* wt = cols + 3 * Ep * Tp;
  uint8_t* live = reinterpret_cast<uint8_t*>(wt + 2 * a.H * Ep);
  const int splits = grad_splits(a.T, a.H, a.E, true), tb = router_grad_row_blocks(a.T);
  const int wt_blocks = a.d_x != nullptr ? a.H / kRgWCols : 0;
  hipLaunchKernelGGL(router_grad_rows_bf16_kernel, dim3(tb + wt_blocks), dim3(kRgRowThreads), 0,
                     s, a.T, a.H, a.E, a.K, a.eps, x, a.pre_gain, a.per_expert_scale, a.logits,
                     a.topk_idx, a.mask, a.d_topk_w, a.d_logits, a.router_w, tb, rows, cols, wt,
                     a.ws_beta, live, a.ws_part_pes);
  const int steps = ((int)(Tp / 32) + splits - 1) / splits;
  const int x_lds = (int)(64 * Ep * 4);
  const bool one = a.d_x != nullptr && grad_one_launch(a.T, a.H, a.E, true);
  auto gw = [&](auto mt, auto masked) {
    constexpr int MT = decltype(mt)::value;
    const int cb = a.H / 64, ey = (a.E + 16 * MT - 1) / (16 * MT), wb = cb * ey * splits;
    const int xb = one ? grad_x_blocks(a.T, a.H, true) : 0;
    const int lds = xb > 0 && x_lds > kRgWBytes ? x_lds : kRgWBytes;
    hipLaunchKernelGGL((router_grad_wx_bf16_kernel<MT, decltype(masked)::value>), dim3(wb + xb),
                       dim3(64 * kRgWaves), lds, s, wb, ey, a.T, a.H, a.E, steps, a.eps, x, live,
                       rows, cols, a.ws_beta, wt, a.router_scale, a.pre_gain, a.ws_part_g,
                       a.ws_part_b, static_cast<bf16*>(a.d_x));
  };
  auto by_mask = [&](auto mt) {
    if (a.mask != nullptr) gw(mt, std::true_type{});
    else gw(mt, std::false_type{});
  };
  // 64 experts a wave: with 128 the parts could be fetched one tile ahead only
  if (a.E <= 32) by_mask(std::integral_constant<int, 2>{});
  else by_mask(std::integral_constant<int, 4>{});
  if (a.d_x != nullptr && !one) {
    const int cb = a.H / 64;
    if (a.E <= 32 * kRgXSteps) {
      const int tiles = (a.T + 15) / 16, want = cb < kRgRound ? kRgRound / cb : 1;
      const int each = (tiles + want - 1) / want;
      const int span = (each + kRgXWaves - 1) / kRgXWaves * kRgXWaves;
      hipLaunchKernelGGL(router_grad_x_loop_kernel, dim3(cb, (tiles + span - 1) / span),
                         dim3(64 * kRgXWaves), 64 * 32 * kRgXSteps * 4 + 512, s, a.T, a.H, a.E,
                         span, a.eps, x, live, rows, a.ws_beta, wt, a.router_scale, a.pre_gain,
                         static_cast<bf16*>(a.d_x));
    } else {
      constexpr int tok = kRgXWaves * kRgXTok;
      hipLaunchKernelGGL(router_grad_x_bf16_kernel, dim3(cb, (a.T + tok - 1) / tok),
                         dim3(64 * kRgXWaves), x_lds, s, a.T, a.H, a.E, a.eps, x, live, rows,
                         a.ws_beta, wt, a.router_scale, a.pre_gain, static_cast<bf16*>(a.d_x));
    }
  }
}

}  // namespace

int balance_blocks(int T) {
  if (T <= kBalOneBlock) return 1;
  const int nb = (T + 63) / 64;
  return nb < kBalMaxBlocks ? nb : kBalMaxBlocks;
}

hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t s) {
  const int nb = balance_blocks(a.T), span = a.T > 0 ? (a.T + nb - 1) / nb : 0;
  by_group(a.E, [&](auto g, auto vec) {
    hipLaunchKernelGGL((balance_partial_kernel<decltype(g)::value, decltype(vec)::value>),
                       dim3(nb), dim3(kBalThreads), 0, s, a.T, a.E, a.K, span, a.logits,
                       a.topk_idx, a.mask, a.balance_coef, a.z_coef, a.ws_part_p, a.ws_part_n,
                       a.ws_part_z, a.ws_part_live, a.loss, a.counts, a.mean_p);
  });
  if (nb > 1)
    hipLaunchKernelGGL(balance_final_kernel, dim3(1), dim3(kBalFinThreads), 0, s, nb, a.E, a.K,
                       a.balance_coef, a.z_coef, a.ws_part_p, a.ws_part_n, a.ws_part_z,
                       a.ws_part_live, a.loss, a.counts, a.mean_p);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceGradArgs& a, hipStream_t s) {
  by_group(a.E, [&](auto g, auto vec) {
    constexpr int per = 256 / decltype(g)::value * kGradUnroll;
    const int nb = (a.T + per - 1) / per;
    hipLaunchKernelGGL((balance_grad_kernel<decltype(g)::value, decltype(vec)::value>), dim3(nb),
                       dim3(256), 0, s, a.T, a.E, a.K, a.logits, a.mask, a.counts, a.loss,
                       a.balance_coef, a.z_coef, a.d_loss, a.d_logits);
  });
  return hipGetLastError();
}

// Workspaces hold as many splits as either type takes: fp32, whose blocks take more
// experts.
int router_grad_max_splits(int T, int H, int E) { return grad_max_splits(T, H, E, false); }

int router_grad_row_blocks(int T) { return (T + 31) / 32 * 32 / kRgTok; }

size_t router_grad_dl_bytes(int T, int H, int E) {
  const size_t Ep = (E + 31) / 32 * 32, Tp = (T + 31) / 32 * 32;
  return 2 * (5 * Tp * Ep + 2 * H * Ep) + Tp;  // more than the 4 T E of fp32
}

hipError_t launch_router_grad(const RouterGradArgs& a, hipStream_t s) {
  if (a.T > 0) {
    if (a.x_bf16) launch_grad_bf16(a, s);
    else launch_grad_f32(a, s);
  }
  constexpr int per = kRgCols / 4;
  const int splits = a.T > 0 ? grad_splits(a.T, a.H, a.E, a.x_bf16) : 0;
  const int row_blocks = a.T > 0 ? router_grad_row_blocks(a.T) : 0;
  auto finish = [&](auto eu) {
    hipLaunchKernelGGL((router_grad_finish_kernel<decltype(eu)::value>),
                       dim3(a.H / kRgCols + (a.E + per - 1) / per), dim3(kRgFinThreads), 0, s,
                       a.H, a.E, splits, row_blocks, a.ws_part_g, a.ws_part_b, a.ws_part_pes,
                       a.router_w, a.router_scale, a.pre_gain, a.d_router_w, a.d_router_scale,
                       a.d_per_expert_scale, a.d_pre_gain);
  };
  if (a.E <= kRgParts) finish(std::integral_constant<int, 1>{});
  else if (a.E <= 2 * kRgParts) finish(std::integral_constant<int, 2>{});
  else finish(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

}  // namespace moe
