// Products in E4M3 with one fp32 scale per block of 128: weights per 128 x 128
// block, activations per 128 consecutive values of a row (quantized on the way
// in).  An 8-bit storage option as on the page "Porting a 128-expert MoE
// (Gemma-4 26B-A4B) to AWS Inferentia2" (section "The fp4 rabbit hole (two of
// them, both dead ends)"), with scales fine enough for both operands to stay
// in 8 bits:
//
//   y_tn = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} xq_tk wq_nk
//
// The inner sum of a 128-block is one v_mfma_f32_16x16x128_f8f6f4 with a zero
// addend; its four results per lane are scaled and added in fp32 registers.
// The weights are the instruction's first operand, so a lane's results are four
// consecutive output columns of ONE token: one scale product per token tile
// and weight block, 4 fused multiply-adds per instruction (16 of its 32 cycles
// on the vector unit, which runs beside the matrix unit).
//
// That instruction does not add in full fp32.  It takes the 128 products in groups
// of eight consecutive k, cuts each product (toward zero) below 2^-13 of the
// largest 2^(ea + eb) of its group, ea and eb the pair's code exponents (-6 for
// subnormal codes), and adds the groups in fp32 (cut at 2^-23): the sums over
// random codes agree with that rule to 2^-22 of their magnitudes.  The other 8-bit
// instructions cut alike; only the bf16 one, at half the rate, does not.  It stays
// for large batches because the codes themselves are rounded at 2^-4.
//
// Operand layout (8-bit, 16 x 128): lane l holds row l % 16 and, with g = l /
// 16, k = 16 g .. 16 g + 15 and k = 64 + 16 g .. 64 + 16 g + 15.  Result: lane
// l, register r is row 4 g + r of the first operand, row l % 16 of the second.
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "wformat.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBlk = 128;              // values that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kInvE4m3Max = 1.0f / 448.0f;  // a block's scale is max |v| times this

__host__ __device__ constexpr int blocks_of(int n) { return (n + kBlk - 1) / kBlk; }

// The sum of 128 products per result, from zero.  Scale operands of 0 select the
// instruction without block scales (the scaled form, with unit scales, ran the
// tiles' inner loop at 0.9 of its rate).
__device__ __forceinline__ f32x4 mfma_blk(i32x8 w, i32x8 x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      w, x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// Magnitudes are compared as their bit patterns: the order is that of the
// numbers, with an infinity and then every NaN above them, so neither is lost as
// in a maximum of floats.
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
template <int CTRL>
__device__ __forceinline__ unsigned dpp_max(unsigned v) {
  return max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}
// Maximum over the 16 lanes of a DPP row, in every lane.
__device__ __forceinline__ unsigned row16_max(unsigned v) {
  v = dpp_max<0xB1>(v);     // lane ^ 1
  v = dpp_max<0x4E>(v);     // lane ^ 2
  v = dpp_max<0x141>(v);    // mirror of 8
  return dpp_max<0x140>(v);
}
// The scale of a block whose largest magnitude is m: NaN, and with it every value
// of the block, where the block holds an infinity or a NaN (an infinite scale
// would leave the others' sign to 448 of either sign).
__device__ __forceinline__ float scale_of(unsigned m) {
  return m < 0x7f800000u ? __uint_as_float(m) * kInvE4m3Max : __uint_as_float(0x7fc00000u);
}

// E4M3 codes of four values already divided by their scale: nearest, ties to
// even; the quotient of the largest value may round past 448 and is clamped.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  auto cl = [](float v) { return fminf(fmaxf(v, -kE4m3Max), kE4m3Max); };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(cl(a), cl(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(cl(c), cl(d), w, true);
}

__device__ __forceinline__ void ld8(const bf16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void ld8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ unsigned amax8(const float (&v)[8]) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag(v[i]));
  return m;
}
// 8 codes of v / s (s = 0 or NaN: zeros).
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float s) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = s > 0.0f ? v[i] / s : 0.0f;
  return make_uint2(encode4(q[0], q[1], q[2], q[3]), encode4(q[4], q[5], q[6], q[7]));
}

// Rows: scale = max |v| * (1 / 448) per 128 values, in fp32, code = E4M3 nearest
// to v / scale (fp32 division: bf16 inputs put many quotients exactly on a
// decision point, where a reciprocal would change the code).  16 lanes a group,
// 8 values a lane.  Memory-bound: 4096 x 2816 in 10.5 us (3.3 TB/s).
template <typename XT, bool PAD>
__global__ __launch_bounds__(256) void quantize_rows128_kernel(long long rows, int cols,
                                                               const XT* __restrict__ in,
                                                               uint8_t* __restrict__ q,
                                                               float* __restrict__ scale) {
  const int nb = blocks_of(cols);
  const long long grp = ((long long)blockIdx.x * 256 + threadIdx.x) / 16;
  if (grp >= rows * nb) return;  // 16 lanes alike
  const int l = threadIdx.x % 16;
  const long long r = grp / nb;
  const int c = (int)(grp % nb) * kBlk + 8 * l;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (c < cols) ld8(in + r * cols + c, v);
  const float s = scale_of(row16_max(amax8(v)));
  if (l == 0) scale[grp] = s;
  const long long pitch = PAD ? (long long)nb * kBlk : cols;
  if (PAD || c < cols) *reinterpret_cast<uint2*>(q + r * pitch + c) = encode8(v, s);
}

// 128 x 128 blocks of [batch, rows, cols]: one workgroup a block, 8 values of 8
// rows a thread.
__global__ __launch_bounds__(256) void quantize_blocks128_kernel(int rows, int cols,
                                                                 const bf16* __restrict__ in,
                                                                 uint8_t* __restrict__ q,
                                                                 float* __restrict__ scale) {
  __shared__ unsigned red[4];
  const int cb = blockIdx.x, rb = blockIdx.y;
  const long long b = blockIdx.z;
  const bf16* src = in + b * rows * cols;
  uint8_t* dst = q + b * rows * cols;
  const int c = cb * kBlk + 8 * (threadIdx.x % 16), r0 = rb * kBlk + threadIdx.x / 16;
  float v[8][8];
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r < rows && c < cols) ld8(src + (long long)r * cols + c, v[i]);
    m = max(m, amax8(v[i]));
  }
  m = row16_max(m);
  m = max(m, (unsigned)__shfl_xor((int)m, 16));
  m = max(m, (unsigned)__shfl_xor((int)m, 32));
  if (lane_id() == 0) red[threadIdx.x / kWave] = m;
  __syncthreads();
  const float s = scale_of(max(max(red[0], red[1]), max(red[2], red[3])));
  if (threadIdx.x == 0) scale[(b * gridDim.y + rb) * gridDim.x + cb] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (r < rows && c < cols)
      *reinterpret_cast<uint2*>(dst + (long long)r * cols + c) = encode8(v[i], s);
  }
}

// Codes times their scale, one rounding: 8 values a thread.
__global__ __launch_bounds__(256) void dequantize_b128_kernel(long long total_rows, int rows,
                                                              int cols, int block_rows,
                                                              const uint8_t* __restrict__ q,
                                                              const float* __restrict__ scale,
                                                              float* __restrict__ out) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int per = cols / 8, nb = blocks_of(cols);
  if (i >= total_rows * per) return;
  const long long r = i / per;
  const int c = 8 * (int)(i % per);
  const long long b = r / rows;
  const int sr = (rows + block_rows - 1) / block_rows;
  const float s = scale[(b * sr + (int)(r % rows) / block_rows) * nb + c / kBlk];
  const uint2 u = *reinterpret_cast<const uint2*>(q + r * cols + c);
  float v[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t lo, hi;
    fp8x4_to_bf16(h == 0 ? u.x : u.y, lo, hi);
    v[4 * h] = __uint_as_float(lo << 16) * s;
    v[4 * h + 1] = __uint_as_float(lo & 0xffff0000u) * s;
    v[4 * h + 2] = __uint_as_float(hi << 16) * s;
    v[4 * h + 3] = __uint_as_float(hi & 0xffff0000u) * s;
  }
  float4* o = reinterpret_cast<float4*>(out + r * cols + c);
  o[0] = make_float4(v[0], v[1], v[2], v[3]);
  o[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// ---------------------------------------------------------------------------
// Shared by both products.
// ---------------------------------------------------------------------------
constexpr int kGateUp = 0, kPlain = 1;

// The tanh form of GELU as z / (1 + exp(-2 u)), u = sqrt(2 / pi) (z + 0.044715
// z^3), on the hardware's exponential and reciprocal (each within an ulp).  No
// cancellation where tanh u nears -1; tanhf had taken half of a gate_up tile's
// time past its products.
__device__ __forceinline__ float gelu_sigmoid(float z) {
  constexpr float c = -2.0f * 0.7978845608028654f * 1.4426950408889634f;  // in powers of 2
  const float u = c * (z + 0.044715f * z * z * z);
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u));
}

__device__ __forceinline__ i32x8 pack8(uint4 a, uint4 b) {
  return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Four consecutive outputs of a row of N columns from column n.  ONCE: fp32 in
// streaming stores (slots, which the combine reads once).
template <bool ONCE = false, typename YT>
__device__ __forceinline__ void store4(YT* __restrict__ row, int n, int N, f32x4 v) {
  if (N % 4 == 0) {
    if (n >= N) return;
    if constexpr (std::is_same<YT, float>::value) {
      if constexpr (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(row + n));
      else *reinterpret_cast<f32x4*>(row + n) = v;
    } else {
      typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
      *reinterpret_cast<bf16x4*>(row + n) =
          bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n + r < N) row[n + r] = from_f32<YT>(v[r]);
}

// ---------------------------------------------------------------------------
// Few rows per group: the weights streamed from HBM into registers once per
// tile of 16 rows.  A block is one row tile x WN waves of NC tiles of 16 columns
// (gate_up: NC gate and the matching NC up tiles), times WK waves that split the
// contraction in 128-blocks and are added through LDS.  Weight loads run NS - 1
// blocks ahead, unconditionally (addresses clamped into their rows), so that a
// step waits for its own slot alone.
//
// The codes are widened to bf16 in registers and multiplied by the bf16
// instruction: the weight stream bounds these kernels, and that instruction adds
// its products to 2^-21 of their magnitudes at most (2^-25 or less in the root mean
// square) where the 8-bit one cuts them as above, 2^-16 at most and 2^-19 for normal
// values (an E4M3 code of h whose sum lies that near a decision point changes).
//
// 26B-A4B at 64 tokens, 113 experts with rows: gate_up 80 us (448 MB, 5.6 TB/s), down
// 55 us (262 MB and 5.8 MB of slots, 4.8 TB/s); at 1 token 11.7 and 6.4 us, the
// latency of one pass over a row.
//
// FUSE: the block quantizes its own rows of x (bf16) or h (fp32) into LDS behind
// the first weight loads, which saves a launch; otherwise their codes and scales
// come from memory with the weights.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  uint4 w;
  fp8x4_to_bf16(lo, w.x, w.y);
  fp8x4_to_bf16(hi, w.z, w.w);
  return __builtin_bit_cast(bf16x8, w);
}
// A lane's 32 codes of a k-block, as loaded: k = 16 g .. + 15, then 64 + 16 g.
struct Codes {
  uint4 a, b;
  __device__ __forceinline__ void load(const uint8_t* row, int kb, int g, int Kd) {
    // (past the row: its first chunk; the other operand is 0 there)
    const int o0 = kb * kBlk + 16 * g, o1 = o0 + 64;
    a = *reinterpret_cast<const uint4*>(row + (o0 < Kd ? o0 : 0));
    b = *reinterpret_cast<const uint4*>(row + (o1 < Kd ? o1 : 0));
  }
  __device__ __forceinline__ void widen(bf16x8 (&v)[4]) const {
    v[0] = widen8(a.x, a.y);
    v[1] = widen8(a.z, a.w);
    v[2] = widen8(b.x, b.y);
    v[3] = widen8(b.z, b.w);
  }
};

constexpr int kFusePad = 16;  // bytes between rows of codes in LDS
__host__ __device__ constexpr int fuse_bytes(int rows, int KB) {
  return rows * (KB * kBlk + kFusePad + 4 * KB);
}

// XT: the type of the rows that FUSE quantizes (void: not fused).
template <int MODE, int WK, int WN, int NC, int NS, typename XT, typename YT>
__global__ __launch_bounds__(64 * WK * WN) void stream_b128_kernel(B128Args a) {
  constexpr bool FUSE = !std::is_same<XT, void>::value;
  constexpr int NW = MODE == kGateUp ? 2 * NC : NC;  // weight tiles per wave
  __shared__ f32x4 red[WK][WN][NW][WK > 1 ? kWave : 1];
  extern __shared__ __align__(16) unsigned char smem[];
  int e, row0, row1, cg;
  const int CG = (a.N + 16 * WN * NC - 1) / (16 * WN * NC);
  if (!stream_item(a.ident, a.rows, a.offsets, a.E, 16, CG, e, row0, row1, cg)) return;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wk = wave % WK, wn = wave / WK;
  const int fr = lane % 16, g = lane / 16;
  const int Kd = a.Kd, KB = blocks_of(Kd), pitch = KB * kBlk;
  const int NR = MODE == kGateUp ? 2 * a.N : a.N;
  const int n0 = (cg * WN + wn) * 16 * NC;
  const uint8_t* wrow[NW];
  const float* wsc[NW];
#pragma unroll
  for (int c = 0; c < NW; ++c) {
    const int first = n0 + 16 * (c % NC), up = c >= NC ? a.N : 0;
    const int r = up + min(first + fr, a.N - 1);
    wrow[c] = a.wq + ((long long)e * NR + r) * Kd;
    wsc[c] = a.wscale +
             ((long long)e * blocks_of(NR) + (up + min(first, a.N - 1)) / kBlk) * KB;
  }
  const int kb0 = wk * KB / WK, kb1 = (wk + 1) * KB / WK, last = max(kb1 - 1, 0);
  Codes rw[NS][NW], rx[NS];
  float sw[NS][NW], sx[NS];
  auto load_w = [&](int kb, int slot) {
#pragma unroll
    for (int c = 0; c < NW; ++c) rw[slot][c].load(wrow[c], kb, g, Kd);
#pragma unroll
    for (int c = 0; c < NW; ++c) sw[slot][c] = wsc[c][kb];
  };
  // a wave without a k-block loads a valid one and never uses it
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    load_w(min(kb0 + s, last), s);
    __builtin_amdgcn_sched_barrier(0);
  }

  const int nrow = row1 - row0;
  const uint8_t* xrow;
  const float* xsc;
  if constexpr (FUSE) {
    uint8_t* xl = smem;
    float* sl = reinterpret_cast<float*>(smem + nrow * (pitch + kFusePad));
    const int l = threadIdx.x % 16;
    for (int k = threadIdx.x / 16; k < nrow * KB; k += 4 * WK * WN) {  // 16 lanes alike
      const int r = k / KB, kb = k % KB, c = kb * kBlk + 8 * l;
      long long t = row0 + r;
      if (MODE == kGateUp) t = a.sorted_slots[t] / a.K;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (c < Kd) ld8(static_cast<const XT*>(a.x) + t * Kd + c, v);
      const float s = scale_of(row16_max(amax8(v)));
      if (l == 0) sl[r * KB + kb] = s;
      *reinterpret_cast<uint2*>(xl + r * (pitch + kFusePad) + c) = encode8(v, s);
    }
    __syncthreads();
    xrow = xl + min(fr, nrow - 1) * (pitch + kFusePad);
    xsc = sl + min(fr, nrow - 1) * KB;
  } else {
    long long t = row0 + min(fr, nrow - 1);
    if (MODE == kGateUp) t = a.sorted_slots[t] / a.K;
    xrow = a.xq + t * pitch;
    xsc = a.xscale + t * KB;
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      rx[s].load(xrow, min(kb0 + s, last), g, pitch);
      sx[s] = xsc[min(kb0 + s, last)];
    }
  }

  f32x4 acc[NW];
#pragma unroll
  for (int c = 0; c < NW; ++c) acc[c] = f32x4{0, 0, 0, 0};
  auto load = [&](int kb, int slot) __attribute__((always_inline)) {
    load_w(kb, slot);
    if constexpr (!FUSE) {
      rx[slot].load(xrow, kb, g, pitch);
      sx[slot] = xsc[kb];
    }
  };
  auto step = [&](int kb, int slot) __attribute__((always_inline)) {
    if constexpr (FUSE) {
      rx[slot].load(xrow, kb, g, pitch);
      sx[slot] = xsc[kb];
    }
    bf16x8 xv[4];
    rx[slot].widen(xv);
#pragma unroll
    for (int c = 0; c < NW; ++c) {
      bf16x8 wv[4];
      rw[slot][c].widen(wv);
      f32x4 d = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[q], xv[q], d, 0, 0, 0);
      const float sc = sx[slot] * sw[slot][c];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[c][r] = __builtin_fmaf(d[r], sc, acc[c][r]);
    }
  };
  int kb = kb0;
  // every load of the unrolled NS steps lies inside the wave's range
  for (; kb + 2 * NS - 2 < kb1; kb += NS) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      load(kb + s + NS - 1, (s + NS - 1) % NS);
      __builtin_amdgcn_sched_barrier(0);
      step(kb + s, s);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  for (; kb < kb1; kb += NS) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (kb + s >= kb1) break;
      if (kb + s + NS - 1 < kb1) load(kb + s + NS - 1, (s + NS - 1) % NS);
      step(kb + s, s);
    }
  }
  if constexpr (WK > 1) {
#pragma unroll
    for (int c = 0; c < NW; ++c) red[wk][wn][c][lane] = acc[c];
    __syncthreads();
  }
  // the WK waves of a column group take its tiles in turn
  const int row = row0 + fr;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (WK > 1 && c % WK != wk) continue;
    const int n = n0 + 16 * c + 4 * g;
    f32x4 v = acc[c], u = {0, 0, 0, 0};
    if constexpr (MODE == kGateUp) u = acc[NC + c];
    if constexpr (WK > 1) {
      v = red[0][wn][c][lane];
      if constexpr (MODE == kGateUp) u = red[0][wn][NC + c][lane];
#pragma unroll
      for (int w = 1; w < WK; ++w) {
        v += red[w][wn][c][lane];
        if constexpr (MODE == kGateUp) u += red[w][wn][NC + c][lane];
      }
    }
    if (row >= row1) continue;
    if constexpr (MODE == kGateUp) {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = gelu_sigmoid(v[r]) * u[r];
      store4(a.h + (size_t)row * a.N, n, a.N, v);
    } else {
      size_t to = row;
      if (!a.ident) {
        to = a.sorted_slots[row];
        v *= a.topk_w[to];
      }
      store4(static_cast<YT*>(a.y) + to * a.N, n, a.N, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows per group: tiles of TM rows x TN weight rows (gate_up: half gate,
// half the matching up rows), WM x WN waves of 16 TI x 16 TJ, on k-tiles of one
// 128-block.  Both operands go global -> LDS directly, a line being a row's 128
// bytes; its 16-byte chunk c sits at position c ^ (line % 8), so the 16 rows
// that a fragment load touches spread over the banks.  The activations have two
// stages: one is refilled once every wave has read it.  The weights have two as
// well where waves share them; where none does (WM = 1) a wave copies its own 64
// rows again as soon as it holds their fragments, into the same lines, and two
// blocks of 256 columns fit into a CU.  The scales of up to KBS k-blocks sit in
// LDS beside the ring, reloaded when those are used up.  A wave multiplies one
// 16-row tile of activations by its TJ weight tiles, and scales the previous
// tile's results meanwhile.
//
// Bound by the matrix cores' power: at 4096 x 4096 x 16384 a k-block of a 256 x
// 256 tile takes 1.7 to 1.9 us on every CU at 1.93 GHz; its products alone take
// 1.1 us (random codes), with the scaling 1.26, and a k-block of a plain E4M3
// library product of 8192^3 1.64.  At 26B-A4B's 4096 tokens gate_up takes 201 us
// (1290 TF/s; weights 507 MB) and down 191 us (254 MB of weights, 369 MB of
// fp32 slots: 3.3 TB/s).
// ---------------------------------------------------------------------------
constexpr int kRowGroup = 4;

template <int WM, int WN, int TI, int TJ>
struct TileShape {
  static constexpr int TM = WM * TI * 16, TN = WN * TJ * 16, NW = WM * WN, THREADS = 64 * NW;
  static constexpr bool OWN_W = WM == 1;                     // no wave shares its weights
  static constexpr int XSTAGE = TM * kBlk, WSTAGE = TN * kBlk;
  static constexpr int XCOPIES = XSTAGE / (THREADS * 16);    // per wave and stage
  static constexpr int WCOPIES = WSTAGE / (THREADS * 16);
  static constexpr int KBS = OWN_W ? 16 : 22;                // even: a run starts in stage 0
  static constexpr int W0 = 2 * XSTAGE;                      // the weights' first line
  static constexpr int SX = W0 + (OWN_W ? 1 : 2) * WSTAGE;   // [KBS][TM]
  static constexpr int SW = SX + KBS * TM * 4;               // [KBS][4]
  static constexpr int TAB = SW + KBS * 4 * 4;               // rtok, slot, weight
  static constexpr int LDS = TAB + 3 * TM * 4;
  static constexpr int HPITCH = TN / 2 + 4;                  // floats
  static_assert(XCOPIES * THREADS * 16 == XSTAGE && WCOPIES * THREADS * 16 == WSTAGE,
                "copies cover a stage");
  static_assert(LDS <= 160 * 1024, "LDS per CU");
};
typedef TileShape<2, 4, 8, 4> WideTile;   // 256 x 256, one block per CU
typedef TileShape<2, 4, 8, 3> Tile192;    // 256 x 192, one block per CU
typedef TileShape<1, 4, 8, 4> PairTile;   // 128 x 256, two blocks per CU
typedef TileShape<2, 2, 4, 4> SmallTile;  // 128 x 128, two blocks per CU
static_assert(PairTile::TM * PairTile::HPITCH * 4 <= PairTile::TAB,
              "h is staged over the ring and the scales");
static_assert(2 * SmallTile::LDS <= 160 * 1024 && 2 * PairTile::LDS <= 160 * 1024,
              "two blocks share a CU");

template <int MODE, int WM, int WN, int TI, int TJ, typename YT>
__global__ __launch_bounds__(64 * WM * WN, 2) void tile_b128_kernel(B128Args a) {
  typedef TileShape<WM, WN, TI, TJ> S;
  constexpr int NS = TJ == 4 ? 2 : TJ;  // weight scales of a wave and k-block
  constexpr int kTM = S::TM, kTN = S::TN, XC = S::XCOPIES, WC = S::WCOPIES;
  constexpr int KBS = S::KBS;
  static_assert(MODE != kGateUp || kTN == 256, "a gate_up tile makes one 128-block of h");
  extern __shared__ __align__(16) unsigned char smem[];
  const int Kd = a.Kd, KB = blocks_of(Kd), N = a.N;
  const int NR = MODE == kGateUp ? 2 * N : N;
  constexpr int COLS = MODE == kGateUp ? kTN / 2 : kTN;  // output columns per tile
  const int NT = (N + COLS - 1) / COLS;
  int e = 0, row0, row1, nt;
  if (a.ident) {
    const int RT = (a.rows + kTM - 1) / kTM;
    const int item = xcd_item(blockIdx.x, RT * NT);
    if (item < 0) return;  // uniform over the block
    // four row tiles at a time, the row tiles fastest: an XCD's run of items
    // then covers few rows and few columns, each read into its L2 once
    const int first = item / (kRowGroup * NT) * kRowGroup, in = item % (kRowGroup * NT);
    const int gr = min(kRowGroup, RT - first);
    nt = in / gr;
    row0 = (first + in % gr) * kTM;
    row1 = min(row0 + kTM, a.rows);
  } else {
    RowTileScan sc;
    row_tile_scan(a.offsets, a.E, kTM, sc);
    const int item = xcd_item(blockIdx.x, sc.total * NT);
    if (item < 0) return;
    weight_major_item(sc, a.offsets, kTM, item, NT, e, row0, row1, nt);
    e = __builtin_amdgcn_readfirstlane(e);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    row1 = __builtin_amdgcn_readfirstlane(row1);
    nt = __builtin_amdgcn_readfirstlane(nt);
  }
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int nbase = nt * COLS;
  float* s_x = reinterpret_cast<float*>(smem + S::SX);
  float* s_w = reinterpret_cast<float*>(smem + S::SW);
  int* rtok = reinterpret_cast<int*>(smem + S::TAB);
  int* row_slot = rtok + kTM;
  float* row_w = reinterpret_cast<float*>(row_slot + kTM);
  if (tid < kTM) {
    const int r = min(row0 + tid, row1 - 1);  // rows past the tile repeat its last: dropped
    rtok[tid] = MODE == kGateUp ? a.sorted_slots[r] / a.K : r;
    if constexpr (MODE == kPlain) {
      const int slot = a.ident ? r : a.sorted_slots[r];
      row_slot[tid] = slot;
      row_w[tid] = a.ident ? 1.0f : a.topk_w[slot];
    }
  }
  __syncthreads();
  const uint8_t* wbase = a.wq + (long long)e * NR * Kd;
  // tile row n of the weights: its row in the expert's matrix (past the last
  // column a valid row, whose outputs are dropped)
  auto wrow = [&](int n) {
    const bool up = MODE == kGateUp && n >= kTN / 2;
    const int col = min(nbase + n - (up ? kTN / 2 : 0), N - 1);
    return col + (up ? N : 0);
  };
  // Copy j of wave w fills lines 8 (NW j + w) .. + 7 of the activations for j <
  // XC, past that 8 lines of the weights from wl(j - XC) on.  Byte offsets from the
  // tile's bases: below 2^32 (a batch's codes of x take 2^30 bytes at most, an
  // expert's weights 2^32).
  // Activation rows end in zeros up to a whole line, so what the weights' part
  // of the last line holds past their row does not matter: their own last
  // chunk, which is a finite number exactly when the output is to be one.
  const int pitch = KB * kBlk;
  const uint8_t* xbase = MODE == kGateUp ? a.xq : a.xq + (long long)row0 * pitch;
  unsigned xsrc[XC], wsrc[WC];
  const int chunk = (lane % 8) ^ (lane / 8);
  // (with one buffer the wave's own)
  auto wl = [&](int j) {
    if (!S::OWN_W) return 8 * (S::NW * j + wave);
    return MODE == kGateUp ? (j / 4) * (kTN / 2) + wn * 32 + 8 * (j % 4) : wn * 64 + 8 * j;
  };
#pragma unroll
  for (int j = 0; j < XC; ++j) {
    const int line = 8 * (S::NW * j + wave) + lane / 8;
    const int row = MODE == kGateUp ? rtok[line] : min(line, row1 - 1 - row0);
    xsrc[j] = (unsigned)row * (unsigned)pitch;
  }
#pragma unroll
  for (int j = 0; j < WC; ++j) wsrc[j] = (unsigned)wrow(wl(j) + lane / 8) * (unsigned)Kd;
  // Copies [j0, j1) of k-block kt, the activations' first (past the last one the
  // last again: bytes that are never read).
  auto copy = [&](int kt, int st, int j0, int j1) __attribute__((always_inline)) {
    const int kc = min(kt, KB - 1) * 8 + chunk;
    const unsigned kx = kc * 16, kw = min(kc, Kd / 16 - 1) * 16;
#pragma unroll
    for (int j = j0; j < j1; ++j) {
      if (j < XC)
        lds_copy16(xbase, xsrc[j] + kx, smem + st * S::XSTAGE + (S::NW * j + wave) * 1024);
      else
        lds_copy16(wbase, wsrc[j - XC] + kw,
                   smem + S::W0 + (S::OWN_W ? 0 : st * S::WSTAGE) + wl(j - XC) * kBlk);
    }
  };
  constexpr int AHEAD = 2;  // copies of a k-block issued before the one before it is done
  // scales of k-blocks [kb0, kb0 + n): activations [kb][256], weights [kb][4]
  // (gate_up: the gate block and the up rows' two; otherwise the two blocks)
  const float* wsbase = a.wscale + (long long)e * blocks_of(NR) * KB;
  const int wblk0 = nbase / kBlk, wblk_up = (N + nbase) / kBlk;
  auto load_scales = [&](int kb0) {
    // all of a thread's loads before the first store: one after the other they
    // had cost 8 us a run
    constexpr int NX = KBS * kTM / (S::THREADS);
    const int n = min(KBS, KB - kb0);
    const int r = tid % kTM, kr = tid / kTM, step = S::THREADS / kTM;
    const float* row = a.xscale + (long long)rtok[r] * KB + kb0;
    float v[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) v[i] = row[min(kr + step * i, n - 1)];
    const int kw = min(tid / 4, n - 1), w = tid % 4;
    const int blk = MODE == kGateUp && w >= 2 ? wblk_up + w - 2 : wblk0 + w;
    const float vw = wsbase[(long long)min(blk, blocks_of(NR) - 1) * KB + kb0 + kw];
#pragma unroll
    for (int i = 0; i < NX; ++i) s_x[(kr + step * i) * kTM + r] = v[i];
    if (tid < KBS * 4) s_w[tid] = vw;
  };
  // this wave's weight tiles: the slots of their scales (of a gate_up wave's two
  // halves; else of its 16-column tiles, none of which crosses a block of 128),
  // fragment offsets
  const int fr = lane % 16, g = lane / 16;
  int ws[NS];
  if constexpr (MODE == kGateUp) {
    ws[0] = 0;  // 128 gate columns from a multiple of 128
    ws[1] = 2 + (N + min(nbase + 32 * wn, N - 32)) / kBlk - wblk_up;
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) ws[i] = (nbase + 16 * (TJ * wn + i * TJ / NS)) / kBlk - wblk0;
  }
  // Lines 16 apart have the same swizzle, so a wave's tiles lie at constants
  // from its first: activations i * 16 lines, weights as wtile().
  const int xline = wm * TI * 16 + fr;
  const int xoff = xline * kBlk + (g ^ (xline & 7)) * 16;
  const int wline = wn * (MODE == kGateUp ? 32 : 16 * TJ) + fr;
  const int woff = wline * kBlk + (g ^ (wline & 7)) * 16;
  auto wtile = [](int j) {
    return (MODE == kGateUp ? (j / 2) * (kTN / 2) + (j % 2) * 16 : j * 16) * kBlk;
  };
  int nv = (row1 - row0 - wm * TI * 16 + 15) / 16;             // tiles of this wave with rows
  nv = __builtin_amdgcn_readfirstlane(max(0, min(TI, nv)));

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  // Fragment at a wave's first tile + at, of the stage at p.
  auto rd = [&](const unsigned char* p, int off, int at) __attribute__((always_inline)) {
    return pack8(*reinterpret_cast<const uint4*>(p + off + at),
                 *reinterpret_cast<const uint4*>(p + (off ^ 64) + at));
  };
  i32x8 fw[TJ], fx[2];
  f32x4 d[2][TJ];
  float sx[2], sw[NS];
  // results of tile i (in d[i & 1]) times their scales
  auto scale_add = [&](int i) __attribute__((always_inline)) {
    float s[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) s[n] = sx[i & 1] * sw[n];
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[i][j][r] = __builtin_fmaf(d[i & 1][j][r], s[j * NS / TJ], acc[i][j][r]);
  };
  auto read_first = [&](int st) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      fw[j] = rd(smem + S::W0 + (S::OWN_W ? 0 : st * S::WSTAGE), woff, wtile(j));
    fx[0] = rd(smem + st * S::XSTAGE, xoff, 0);
  };
  // One k-block from stage `st`, its weight fragments in fw and its first
  // activation tile in fx[0]; kl: its place among the staged scales.
  // Activation tiles are read one ahead.  Before the last tile's products comes
  // the block's barrier: past it the stage is free for k-block kt + 2 (every
  // wave has its last fragments) and k-block kt + 1 has landed everywhere, so
  // its first fragments are read behind those products.  No branch: one would
  // let the compiler move products past it and their operands would pile up.
  auto block = [&](int kt, int kl, auto st_tag, auto ti_tag) __attribute__((always_inline)) {
    constexpr int st = decltype(st_tag)::value;
    constexpr int TV = decltype(ti_tag)::value;
#pragma unroll
    for (int n = 0; n < NS; ++n) sw[n] = s_w[kl * 4 + ws[n]];
#pragma unroll
    for (int i = 0; i < TV; ++i) {
      sx[i & 1] = s_x[kl * kTM + xline + 16 * i];
      if (i + 1 < TV) {
        fx[(i + 1) & 1] = rd(smem + st * S::XSTAGE, xoff, (i + 1) * 16 * kBlk);
      } else {
        wait_lds();
        wait_vmem<0>();
        block_barrier();
        copy(kt + 2, st, 0, AHEAD);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) d[i & 1][j] = mfma_blk(fw[j], fx[i & 1]);
      if (i + 1 == TV) {
        __builtin_amdgcn_sched_barrier(0);
        read_first(1 - st);  // (past the end: never used)
        __builtin_amdgcn_sched_barrier(0);
      }
      // the other copies in three parts; the products above have waited for the
      // weights' fragments, so a wave's own lines are free
      if (S::OWN_W && i == 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        if (i == (TV >= 4 ? p * TV / 8 : 0))
          copy(kt + 1, 1 - st, AHEAD + p * (XC + WC - AHEAD) / 3,
               AHEAD + (p + 1) * (XC + WC - AHEAD) / 3);
      if (i > 0) scale_add(i - 1);
      __builtin_amdgcn_sched_barrier(0);  // no fragment is read further ahead
    }
    scale_add(TV - 1);
  };
  auto loop = [&](auto ti_tag) __attribute__((always_inline)) {
    for (int k0 = 0; k0 < KB; k0 += KBS) {
      if (k0 > 0) {
        __syncthreads();  // the scales of the k-blocks before are used up
        load_scales(k0);
        __syncthreads();
      }
      const int n = min(KBS, KB - k0);
      for (int kl = 0; kl < n; kl += 2) {
        block(k0 + kl, kl, std::integral_constant<int, 0>{}, ti_tag);
        if (kl + 1 < n) block(k0 + kl + 1, kl + 1, std::integral_constant<int, 1>{}, ti_tag);
      }
    }
  };
  copy(0, 0, 0, XC + WC);
  load_scales(0);
  wait_vmem<0>();
  __syncthreads();
  copy(1, 1, 0, AHEAD);
  read_first(0);
  // as many tiles as hold the wave's rows (every wave takes part in the copies
  // and barriers)
  if (TI > 4 && nv > 4) loop(std::integral_constant<int, TI>{});
  else if (nv > 2) loop(std::integral_constant<int, 4>{});
  else loop(std::integral_constant<int, 2>{});
  wait_vmem<0>();
  __syncthreads();

  if constexpr (MODE == kGateUp) {
    // h = GELU(gate) * up in fp32, staged row-major; then 128 columns of a row
    // share a scale: 4 lanes a row, 32 columns a lane
    float* hs = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      if (i >= nv) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = wn * 32 + 16 * j + 4 * g;
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[r] = nbase + c + r < N ? gelu_sigmoid(acc[i][j][r]) * acc[i][2 + j][r] : 0.0f;
        *reinterpret_cast<f32x4*>(hs + (xline + 16 * i) * S::HPITCH + c) = v;
      }
    }
    __syncthreads();
    const int nbh = blocks_of(N);
#pragma unroll
    for (int it = 0; it < kTM * 4 / (S::THREADS); ++it) {
      const int k = tid + it * S::THREADS, r = k / 4, c = 32 * (k % 4);
      const bool on = row0 + r < row1;
      float v[32];
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(hs + r * S::HPITCH + c + 4 * i);
        v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) m = max(m, mag(v[i]));
      const float s = scale_of(dpp_max<0x4E>(dpp_max<0xB1>(m)));
      // one division a row: h is an fp32 sum already, no decision point is hit
      // exactly, and an ulp of the quotient moves no more codes than one of h.  A
      // scale that is no normal number has no reciprocal in fp32 (0 times infinity
      // would make a NaN of every zero): there the quotients themselves
      if (s >= 0x1p-126f) {
        const float inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= inv;
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = s > 0.0f ? v[i] / s : 0.0f;
      }
      if (!on) continue;  // columns past the last are zeros: the row's padding
      uint32_t q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i] = encode4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      uint4* dst = reinterpret_cast<uint4*>(a.hq + (size_t)(row0 + r) * (nbh * kBlk) + nbase + c);
      dst[0] = make_uint4(q[0], q[1], q[2], q[3]);
      dst[1] = make_uint4(q[4], q[5], q[6], q[7]);
      if (c == 0) a.hscale[(size_t)(row0 + r) * nbh + nbase / kBlk] = s;
    }
  } else {
    // through LDS, 128 rows at a time, so that a wave stores whole rows of the
    // tile (as the results lie, 64 bytes of 16 rows: the stores of fp32 slots
    // took twice the time)
    constexpr int PITCH = kTN + 4, ROWS = S::OWN_W ? 64 : 128, CH = kTN / 4;
    static_assert(ROWS * PITCH * 4 <= S::TAB, "results are staged over the ring and the scales");
    float* ys = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int pass = 0; pass < kTM / ROWS; ++pass) {
      if (pass > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        if (i < nv && (wm * TI + i) * 16 / ROWS == pass) {
          float* row = ys + ((wm * TI + i) * 16 % ROWS + fr) * PITCH + wn * 16 * TJ + 4 * g;
#pragma unroll
          for (int j = 0; j < TJ; ++j) *reinterpret_cast<f32x4*>(row + 16 * j) = acc[i][j];
        }
      }
      __syncthreads();
#pragma unroll 4
      for (int k = tid; k < ROWS * CH; k += S::THREADS) {
        const int r = k / CH, c = 4 * (k % CH), rr = pass * ROWS + r;
        if (row0 + rr >= row1) break;
        const f32x4 v = *reinterpret_cast<const f32x4*>(ys + r * PITCH + c);
        store4<true>(static_cast<YT*>(a.y) + (size_t)row_slot[rr] * N, nbase + c, N,
                     v * row_w[rr]);
      }
    }
  }
}

template <int MODE, int WK, int WN, int NC, int NS, typename XT, typename YT>
hipError_t launch_stream(const B128Args& a, hipStream_t s) {
  const long long cgs = (a.N + 16 * WN * NC - 1) / (16 * WN * NC);
  const long long grid = cgs * tile_count_bound(a.ident, a.rows, a.T, a.E, 16);
  const int lds = std::is_same<XT, void>::value
                      ? 0 : fuse_bytes(a.T < 16 ? a.T : 16, blocks_of(a.Kd));
  hipLaunchKernelGGL((stream_b128_kernel<MODE, WK, WN, NC, NS, XT, YT>), dim3((unsigned)grid),
                     dim3(64 * WK * WN), lds, s, a);
  return hipGetLastError();
}

template <int MODE, int WM, int WN, int TI, int TJ, typename YT>
hipError_t launch_tile(const B128Args& a, hipStream_t s) {
  typedef TileShape<WM, WN, TI, TJ> S;
  auto kf = tile_b128_kernel<MODE, WM, WN, TI, TJ, YT>;
  // set on every call: the attribute belongs to the current device
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kf),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
  if (e != hipSuccess) return e;
  const int COLS = MODE == kGateUp ? S::TN / 2 : S::TN;
  const long long grid = (long long)tile_count_bound(a.ident, a.rows, a.T, a.E, S::TM) *
                         ((a.N + COLS - 1) / COLS);
  hipLaunchKernelGGL(kf, dim3((unsigned)grid), dim3(S::THREADS), S::LDS, s, a);
  return hipGetLastError();
}
template <typename S>
struct Launch;
template <int WM, int WN, int TI, int TJ>
struct Launch<TileShape<WM, WN, TI, TJ>> {
  static hipError_t plain(const B128Args& a, bool y_bf16, hipStream_t s) {
    return y_bf16 ? launch_tile<kPlain, WM, WN, TI, TJ, bf16>(a, s)
                  : launch_tile<kPlain, WM, WN, TI, TJ, float>(a, s);
  }
  static hipError_t gate_up(const B128Args& a, hipStream_t s) {
    return launch_tile<kGateUp, WM, WN, TI, TJ, float>(a, s);
  }
};

template <typename XT, bool PAD>
hipError_t quantize_rows(long long rows, int cols, const void* x, uint8_t* q, float* scale,
                         hipStream_t s) {
  const long long lanes = rows * blocks_of(cols) * 16;
  hipLaunchKernelGGL((quantize_rows128_kernel<XT, PAD>), dim3((unsigned)((lanes + 255) / 256)),
                     dim3(256), 0, s, rows, cols, static_cast<const XT*>(x), q, scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_b128(int block_rows, long long batch, int rows, int cols, const void* w,
                                uint8_t* q, float* scale, hipStream_t s) {
  if (block_rows == 1) return quantize_rows<bf16, false>(batch * rows, cols, w, q, scale, s);
  // the grid's z axis holds 65535 matrices at a time
  const int rb = blocks_of(rows), cb = blocks_of(cols);
  for (long long b = 0; b < batch; b += 65535) {
    const unsigned nz = (unsigned)(batch - b < 65535 ? batch - b : 65535);
    hipLaunchKernelGGL(quantize_blocks128_kernel, dim3(cb, rb, nz), dim3(256), 0, s, rows, cols,
                       static_cast<const bf16*>(w) + b * rows * cols, q + b * rows * cols,
                       scale + b * rb * cb);
  }
  return hipGetLastError();
}

hipError_t launch_dequantize_b128(int block_rows, long long batch, int rows, int cols,
                                  const uint8_t* q, const float* scale, float* out,
                                  hipStream_t s) {
  const long long n = batch * rows * (cols / 8);
  hipLaunchKernelGGL(dequantize_b128_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                     batch * rows, rows, cols, block_rows, q, scale, out);
  return hipGetLastError();
}

// Streaming where an expert's rows fill one 16-row tile on average, or where
// reading the weights again for every further tile costs little: at most 96 MB
// (8 experts of 2816 x 704, top 8: 24 tokens 35 us streamed, 43 tiled; 64 tokens
// 51 and 45; of 1024 x 256, top 4: 256 tokens 27 and 34).  What decides is the rows
// per expert, which the limit of 256 tokens stands for: experts of 2816 x 704, us
// streamed and tiled,
//   128, top 8: 32 tokens 106 138, 64 135 161, 128 (8 rows an expert) 157 166, 160
//     177 174, 200 191 176, 256 (16 rows) 209 177;
//   128, top 2: 256 tokens (4 rows) 132 157, 400 140 158, 600 (9 rows) 168 170;
//   256, top 4: 256 tokens (4 rows) 240 258, 400 270 269, 512 (8 rows) 311 284.
// Past eight rows an expert the limit is late, below it early for few slots a token:
// up to 18 % of the call.
bool b128_streams(int T, int rows, int E, int H, int I) {
  const long long again = (long long)E * ((rows + 16 * E - 1) / (16 * E) - 1) * 3 * H * I;
  return T <= kB128StreamTokens && again <= 96LL << 20;
}

// The tiles of a product of one group, by the rounds of blocks that each shape
// needs.  A round of 256 tiles of 256 x 256 takes some 8 units, of 256 x 192 6.4, of
// 512 small ones (two per CU) 5, and one of at most 256 small ones 3.3 (2112-long
// rows, 2816 columns, 1024 / 2048 / 4096 / 8192 tokens: small 25 / 33 / 53 / 82 us,
// 192 columns 33 / 35 / 40 / 73, 256 columns 38 / 41 / 46 / 82; 4096 x 4096 x 4096
// 94, 109, 80).  The order hardly depends on the contraction: of the three shapes
// forced on 60 products (rows of 512, 1408, 2112, 5632, 16384 values; 2112, 2816,
// 4096 columns; 1024 to 8192 tokens) the one chosen was the fastest or within 3 %.
enum class Tile { kSmall, k192, kWide };
static Tile linear_tile(long long rows, long long cols) {
  auto tiles = [&](int tm, int tn) { return (rows + tm - 1) / tm * ((cols + tn - 1) / tn); };
  const long long small = tiles(128, 128), rest = small % 512;
  const double s = 5.0 * (small / 512) + (rest == 0 ? 0.0 : rest <= 256 ? 3.3 : 5.0);
  const double m = 6.4 * ((tiles(256, 192) + 255) / 256);
  const double w = 8.0 * ((tiles(256, 256) + 255) / 256);
  return s < m && s < w ? Tile::kSmall : m < w ? Tile::k192 : Tile::kWide;
}

// Whether the streaming blocks quantize their own rows: few enough of them that
// the repeated work costs less than the launch it saves (T <= most), and their
// codes fit in LDS beside the partial sums (48 KB).  26B-A4B gate_up: experts at
// 4 / 8 / 16 tokens 44 / 67 / 101 us fused, 51 / 67 / 94 us not; a 2112 x 2816
// product at 8 / 16 tokens 11.1 / 17.5 and 11.3 / 10.8 us.  down's rows are short
// (704 values): fused at every streamed size (64 tokens 60 -> 55 us with the
// quantizer).
constexpr int kFuseGateUpTokens = 4, kFuseLinearTokens = 8;
static bool fuses(int T, int Kd, int most) {
  return T <= most && fuse_bytes(T < 16 ? T : 16, blocks_of(Kd)) <= 48 * 1024;
}

template <typename XT>
static hipError_t stream_linear(const B128Args& a, bool y_bf16, hipStream_t s) {
  return y_bf16 ? launch_stream<kPlain, 4, 1, 1, 3, XT, bf16>(a, s)
                : launch_stream<kPlain, 4, 1, 1, 3, XT, float>(a, s);
}

// x quantized, y = x W^T.
hipError_t launch_linear_b128(const B128Args& a, const void* x, uint8_t* xq, float* xscale,
                              bool y_bf16, hipStream_t s) {
  if (fuses(a.rows, a.Kd, kFuseLinearTokens)) {
    B128Args f = a;
    f.x = x;
    return stream_linear<bf16>(f, y_bf16, s);
  }
  hipError_t e = quantize_rows<bf16, true>(a.rows, a.Kd, x, xq, xscale, s);
  if (e != hipSuccess) return e;
  // streamed while there is one row tile, or all of them together read at most 64
  // MB of weights (2112 x 2816: 128 tokens 16.4 us streamed, 20.8 tiled, 256 tokens
  // 30.4 and 25.0; 4096 x 4096: 64 tokens 23.9 and 26.6; 4096 x 16384: 16 tokens
  // 24.4 and 30.6, 32 tokens 41.8 and 31.2; 8192 x 8192: 16 tokens 23.5 and 52.6)
  if (a.rows <= 16 || (a.rows + 15LL) / 16 * a.N * a.Kd <= 64LL << 20)
    return stream_linear<void>(a, y_bf16, s);
  switch (linear_tile(a.rows, a.N)) {
    case Tile::kSmall: return Launch<SmallTile>::plain(a, y_bf16, s);
    case Tile::k192: return Launch<Tile192>::plain(a, y_bf16, s);
    default: return Launch<WideTile>::plain(a, y_bf16, s);
  }
}

// Four waves of one column tile, two k-blocks deep (26B-A4B at 64 tokens: 54.6
// us; two tiles a wave 54.4, deeper rings 55 to 60, eight waves 55.9).
template <typename XT>
static hipError_t stream_down(const B128Args& a, bool y_bf16, hipStream_t s) {
  return y_bf16 ? launch_stream<kPlain, 1, 4, 1, 2, XT, bf16>(a, s)
                : launch_stream<kPlain, 1, 4, 1, 2, XT, float>(a, s);
}

// x quantized; h = GELU(gate) * up, quantized; y = topk_w * down h.  gu and dn
// are the two products' arguments.
hipError_t launch_expert_ffn_b128(const B128Args& gu, const B128Args& dn, const void* x,
                                  uint8_t* xq, float* xscale, bool y_bf16, hipStream_t s) {
  hipError_t e;
  if (b128_streams(gu.T, gu.rows, gu.E, gu.Kd, gu.N)) {
    B128Args f = gu;
    f.x = x;
    if (fuses(gu.T, gu.Kd, kFuseGateUpTokens)) {
      // eight waves a block where the blocks do not fill the CUs (1 token: 13.4 ->
      // 11.7 us), else four (4 tokens: 51 -> 44 us with down and combine)
      const long long blocks = (long long)tile_count_bound(false, gu.rows, gu.T, gu.E, 16) *
                               ((gu.N + 31) / 32);
      e = blocks <= 256 ? launch_stream<kGateUp, 8, 1, 2, 3, bf16, float>(f, s)
                        : launch_stream<kGateUp, 4, 1, 2, 2, bf16, float>(f, s);
    } else {
      if ((e = quantize_rows<bf16, true>(gu.T, gu.Kd, x, xq, xscale, s)) != hipSuccess) return e;
      e = launch_stream<kGateUp, 4, 1, 2, 2, void, float>(gu, s);
    }
    if (e != hipSuccess) return e;
    if (fuses(dn.T, dn.Kd, kB128StreamTokens)) {
      B128Args h = dn;
      h.x = gu.h;
      return stream_down<float>(h, y_bf16, s);
    }
    if ((e = quantize_rows<float, true>(gu.rows, gu.N, gu.h, gu.hq, gu.hscale, s)) != hipSuccess)
      return e;
    return stream_down<void>(dn, y_bf16, s);
  }
  if ((e = quantize_rows<bf16, true>(gu.T, gu.Kd, x, xq, xscale, s)) != hipSuccess) return e;
  // tiles of 128 rows: an expert's last one wastes less than of 256 (experts and
  // combine at 300 / 1024 / 2048 / 4096 / 8192 tokens 194 / 242 / 324 / 472 / 820
  // us, with 256 rows 209 / 257 / 342 / 483 / 833, down alike)
  if ((e = Launch<PairTile>::gate_up(gu, s)) != hipSuccess) return e;
  // down: 256 rows a tile once an expert has some 192 on average (experts and
  // combine at 512 / 1024 / 2560 / 4096 / 8192 tokens 224 / 250 / 353 / 470 / 820 us,
  // with 128 rows 206 / 239 / 343 / 481 / 851)
  return dn.rows < 192LL * dn.E ? Launch<PairTile>::plain(dn, y_bf16, s)
                                : Launch<WideTile>::plain(dn, y_bf16, s);
}

}  // namespace moe
