// Backward pass of the gated feed-forward block (the experts and the dense MLP
// of the page "Porting a 128-expert MoE (Gemma-4 26B-A4B) to AWS Inferentia2",
// section "The architecture: a dual-path FFN nobody warned me about").
//
// Forward, for a row r (a token-slot of an expert, or a token of the dense MLP)
// with input x, routing weight w (1 for the dense MLP) and kept projections
// g = W_g x, u = W_u x:
//   h = gelu(g) * u,   y = w W_d h.
// Backward, from the gradient d of y summed over the slots of a token:
//   v   = W_d^T d                                (DU, contraction over H)
//   d_w = <v, h>
//   d_g = w v u gelu'(g),  d_u = w v gelu(g)     (DU's epilogue)
//   d_x = W_g^T d_g + W_u^T d_u, summed over a token's slots  (DX, over 2 I)
//   d_W_gu = sum_r [d_g, d_u]_r x_r^T            (DWGU, over the expert's rows)
//   d_W_d  = sum_r d_r (w h)_r^T                 (DWDN, over the expert's rows)
// Four grouped matrix products of 2 (S H I) to 4 (S H I) operations each, S rows.
//
// d_w comes from <v, h>, not from <d, W_d h>: it needs no expert output kept.
// Rows are the expert-sorted slots of the dispatch; row_tok maps a row to its
// token, -1 where the token does not count: such a row enters every product as
// zeros (read from a page of zeros), whatever its token's data hold.
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

enum Kind { kDU = 0, kDX = 1, kDWGU = 2, kDWDN = 3 };

// A row of zeros as long as the widest operand row.
__device__ const uint4 zero_row[8192 * 2 / 16] = {};

// h, and with v = W_d^T d the gradients of the gate and of the up projection
// (without the routing weight).  gelu(z) = z s(z), s the logistic function of
// q = 2 c (z + a z^3): (1 + tanh(q / 2)) / 2 = s, so nothing cancels where the
// tanh is near -1.  Past |z| = 64 s is 0 or 1 to the last bit, so z is clamped
// there inside the polynomial: z^3 cannot overflow into inf * 0.
template <bool FAST>
__device__ __forceinline__ void act_grad(float z, float up, float v, float& h, float& dg,
                                         float& du) {
  const float c2 = 1.5957691216057308f, a = 0.044715f;  // 2 sqrt(2 / pi)
  const float zc = fminf(fmaxf(z, -64.0f), 64.0f), z2 = zc * zc;
  const float q = c2 * zc * (1.0f + a * z2);
  const float e = FAST ? __expf(-q) : expf(-q);
  const float s = 1.0f / (1.0f + e);
  const float gelu = z * s;
  const float slope = s + gelu * (1.0f - s) * c2 * (1.0f + 3.0f * a * z2);
  h = gelu * up;
  dg = v * up * slope;
  du = v * gelu;
}

// Row r of the sorted order -> its token, -1 if the token does not count; slot ->
// its row.  A slot that the dispatch dropped keeps whatever the workspace held:
// readers of slot_row check that sorted_slots points back.
__global__ __launch_bounds__(256) void rows_kernel(int rows, int ident, int E, int K,
                                                   const int32_t* __restrict__ offsets,
                                                   const int32_t* __restrict__ sorted_slots,
                                                   const uint8_t* __restrict__ mask,
                                                   int32_t* __restrict__ row_tok,
                                                   int32_t* __restrict__ slot_row) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= (ident ? rows : offsets[E])) return;
  int tok = r;
  if (!ident) {
    const int slot = sorted_slots[r];
    slot_row[slot] = r;
    tok = slot / K;
  }
  row_tok[r] = mask && !mask[tok] ? -1 : tok;
}

// d_x[t] = sum over t's slots (k ascending) of their rows of d_xs, in fp32;
// d_topk_w[t, k] = the sum of its row's partial sums (column tiles ascending).
template <typename XT>
__global__ __launch_bounds__(256) void combine_grad_kernel(
    int T, int H, int K, int E, int parts, long long part_stride,
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ sorted_slots,
    const int32_t* __restrict__ slot_row, const XT* __restrict__ d_xs,
    const float* __restrict__ part, XT* __restrict__ d_x, float* __restrict__ d_topk_w) {
  __shared__ int row_of[256];
  const int t = blockIdx.x;
  const int total = offsets[E];
  for (int k = threadIdx.x; k < K; k += 256) {
    const int slot = t * K + k;
    int r = slot_row[slot];
    if (r < 0 || r >= total || sorted_slots[r] != slot) r = -1;  // a dropped slot
    row_of[k] = r;
    if (d_topk_w) {
      float s = 0.0f;
      if (r >= 0)
        for (int p = 0; p < parts; ++p) s += part[p * part_stride + r];
      d_topk_w[slot] = s;
    }
  }
  if (!d_x) return;
  __syncthreads();
  for (int c = threadIdx.x * 8; c < H; c += 256 * 8) {
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int k0 = 0; k0 < K; k0 += 8) {
      XT v[8][8];
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int r = k0 + kk < K ? row_of[k0 + kk] : -1;
        if (r >= 0) {
          const uint4* q = reinterpret_cast<const uint4*>(d_xs + (size_t)r * H + c);
#pragma unroll
          for (int i = 0; i < (int)(sizeof(XT) / 2); ++i)
            reinterpret_cast<uint4*>(v[kk])[i] = q[i];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[kk][j] = (XT)0.0f;
        }
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += to_f32(v[kk][j]);
    }
    XT o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = from_f32<XT>(acc[j]);
    uint4* q = reinterpret_cast<uint4*>(d_x + (size_t)t * H + c);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(XT) / 2); ++i) q[i] = reinterpret_cast<uint4*>(o)[i];
  }
}

// Operands of one product; which are used depends on the kind.
struct Operands {
  int H, I, E, K, rows, ident;
  const int32_t* offsets;
  const int32_t* row_tok;
  const int32_t* sorted_slots;
  const float* topk_w;
  const void* x;        // [T, H]
  const void* d_out;    // [T, H]
  const void* kept;     // [rows, 2 I]
  const void* w_gate;   // DX: group 0's [I, H] gate rows
  const void* w_up;
  const void* w_down;   // DU: group 0's [H, I]
  long long gu_stride, dn_stride;
  void* d_gu;           // [rows, 2 I]
  void* hw;             // [rows, I]
  float* part;          // [column tiles, rows]
  void* d_xs;           // DX: [rows, H]
  void* d_gate;         // DWGU: group 0's [I, H] gate rows
  void* d_up;
  void* d_down;         // DWDN: group 0's [H, I]
};

// ---------------------------------------------------------------------------
// bf16: tiles of 256 x 256 on v_mfma_f32_32x32x16_bf16
// ---------------------------------------------------------------------------
// Two forms of an operand in LDS, per k-tile of 32:
//  - "row": memory rows run along k (the gathered rows of DU and DX).  256 rows
//    of 64 B, 16-B chunk c of row r at position c ^ ((r >> 2) & 3); a fragment is
//    one 16-B read.
//  - "col": memory rows are the k index (weights of DU and DX, both operands of
//    the weight gradients).  32 rows of 512 B, 32-B piece p of row k at position
//    p ^ (2 (k & 3)); a fragment is two transposing 8-B reads
//    (ds_read_b64_tr_b16: each group of 16 lanes reads four k of 16 columns, lane
//    i gets column i).  The four k of a group lie in four pieces and the next
//    group's four in the other four of the same 256 B: no bank twice.
// Both come in by direct global -> LDS copies into a ring of stages.  The B
// columns are the instruction's first operand, so a lane's results are runs of
// four consecutive columns of one row.
constexpr int BT = 256, GK = 32;
constexpr int kOpBytes = BT * GK * 2;         // one operand's k-tile
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kStages = 4;
constexpr int kTab = 2048;                    // rows whose tokens are in LDS at a time
constexpr int kStageRows = 128, kF32Pitch = BT + 4, kBfPitch = BT + 8;
constexpr int kStagingBytes = kStageRows * kF32Pitch * 4;
constexpr int kRingBytes = kStages * kStageBytes > kStagingBytes ? kStages * kStageBytes
                                                                 : kStagingBytes;
constexpr int kLdsBytes = kRingBytes + kTab * 4;
static_assert(BT * kBfPitch * 2 <= kLdsBytes && kLdsBytes <= 160 * 1024, "LDS");

__device__ __forceinline__ int rswz(int r, int c) { return c ^ ((r >> 2) & 3); }
__device__ __forceinline__ int cswz(int k, int p) { return p ^ ((k & 3) << 1); }

template <int KIND, typename WT>
__global__ __launch_bounds__(512, 1) void grad_gemm_kernel(Operands o, int MT, int NT) {
  constexpr bool DW = KIND == kDWGU || KIND == kDWDN;
  constexpr int WN = 4, NW = 8, LPW = kStageBytes / 1024 / NW;  // copies a wave and k-tile
  constexpr int TM = 4, TN = 2, NF = TM + TN, NMF = TM * TN;
  constexpr int WR = 32 * TM, WC = 32 * TN;
  extern __shared__ __align__(16) unsigned char smem[];
  int* tab = reinterpret_cast<int*>(smem + kRingBytes);

  const int H = o.H, I = o.I;
  const int Nout = KIND == kDU || KIND == kDWDN ? I : H;
  int e = 0, row0, row1, mt = 0, nt;
  if constexpr (DW) {
    const int item = xcd_item(blockIdx.x, o.E * MT * NT);
    if (item < 0) return;  // uniform over the block
    e = item / (MT * NT);
    mt = item / NT % MT;
    nt = item % NT;
    const bool all = o.ident || o.rows == 0;  // no rows: the offsets may not exist
    row0 = all ? 0 : o.offsets[e];
    row1 = all ? o.rows : o.offsets[e + 1];
  } else {
    RowTileScan sc;
    int R;
    if (o.ident) {
      R = (o.rows + BT - 1) / BT;
    } else {
      row_tile_scan(o.offsets, o.E, BT, sc);
      R = sc.total;
    }
    const int item = xcd_item(blockIdx.x, R * NT);
    if (item < 0) return;
    if (o.ident) {
      nt = item % NT;
      row0 = item / NT * BT;
      row1 = min(row0 + BT, o.rows);
    } else {
      weight_major_item(sc, o.offsets, BT, item, NT, e, row0, row1, nt);
    }
  }
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int m0 = mt * BT, n0 = nt * BT;
  const bf16* zeros = reinterpret_cast<const bf16*>(zero_row);

  // Sources of this lane's copies.  Copies 0 .. 15 of a stage are A, 16 .. 31 B.
  const bf16* src[LPW];   // row form: + 32 per k-tile; col form: the first k row
  int kr[LPW];            // col form: this lane's k row of the tile
  const int M = KIND == kDWGU ? 2 * I : H;  // DW: rows of the output
  const bool waveA = wave < NW / 2;
#pragma unroll
  for (int j = 0; j < LPW; ++j) {
    const int q = (wave * LPW + j) % (NW * LPW / 2);
    if (!DW && waveA) {
      const int r = 16 * q + lane / 4;
      int gr = row0 + r;
      if (gr >= row1) gr = row0;  // past the tile: a valid row, output dropped
      const bf16* p;
      if constexpr (KIND == kDU) {
        const int tok = o.row_tok[gr];
        p = tok < 0 ? zeros : static_cast<const bf16*>(o.d_out) + (size_t)tok * H;
      } else {
        p = static_cast<const bf16*>(o.d_gu) + (size_t)gr * 2 * I;
      }
      src[j] = p + rswz(r, lane % 4) * 8;
      kr[j] = 0;
    } else {
      kr[j] = 2 * q + lane / 32;
      const int piece = cswz(kr[j], (lane % 32) / 2);
      int c = (DW && waveA ? m0 : n0) + piece * 16 + (lane & 1) * 8;
      if (c >= (DW && waveA ? M : Nout)) c = 0;  // a valid column, output dropped
      if constexpr (KIND == kDU) {
        src[j] = static_cast<const bf16*>(o.w_down) + (size_t)e * o.dn_stride +
                 (size_t)kr[j] * I + c;
      } else if constexpr (KIND == kDX) {
        src[j] = static_cast<const bf16*>(o.w_gate) + (size_t)e * o.gu_stride +
                 (size_t)kr[j] * H + c;
      } else if constexpr (KIND == kDWGU) {
        src[j] = (waveA ? static_cast<const bf16*>(o.d_gu) : static_cast<const bf16*>(o.x)) + c;
      } else {
        src[j] = (waveA ? static_cast<const bf16*>(o.d_out) : static_cast<const bf16*>(o.hw)) + c;
      }
    }
  }
  // the up rows' distance from where the gate rows would go on
  const long long up_shift =
      KIND == kDX ? static_cast<const bf16*>(o.w_up) -
                        (static_cast<const bf16*>(o.w_gate) + (size_t)I * H)
                  : 0;

  // Fragment byte offsets within a stage, per k16 half s.
  const int fr = lane % 32, fq = lane / 32;
  auto row_off = [&](int r, int s) { return r * 64 + rswz(r, 2 * s + fq) * 16; };
  // col form: k = 16 s + 8 fq + (lane % 16) / 4 (+ 4 for the second read),
  // columns c .. c + 3 of the lane's address
  const int tk = 8 * fq + (lane % 16) / 4, tc = 16 * ((lane / 16) % 2) + 4 * (lane % 4);
  auto col_off = [&](int c, int k) {
    c += tc;
    return k * (BT * 2) + cswz(k, c / 16) * 32 + (c % 16) * 2;
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  bf16x8 f0[NF], f1[NF];
  int offA[TM], offB[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
    offA[i] = DW ? col_off(wm * WR + i * 32, tk) : row_off(wm * WR + i * 32 + fr, 0);
#pragma unroll
  for (int j = 0; j < TN; ++j) offB[j] = kOpBytes + col_off(wn * WC + j * 32, tk);
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  auto rd_col = [&](const unsigned char* p) {
    union {
      s16x4 h[2];
      bf16x8 v;
    } u;
#if defined(__HIP_DEVICE_COMPILE__)
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * BT * 2));
#else
    u.v = bf16x8{};
#endif
    return u.v;
  };
  // k rows 16 s + tk: the swizzle depends on k & 3 = tk & 3 alone, so half s is
  // 16 rows further on; the row form's half 1 flips chunk bit 1
  auto rd = [&](const unsigned char* st, int s, int f, bf16x8 (&d)[NF]) {
    if (f < TM) {
      if constexpr (DW)
        d[f] = rd_col(st + offA[f] + s * 16 * BT * 2);
      else
        d[f] = *reinterpret_cast<const bf16x8*>(st + (offA[f] ^ (s * 32)));
    } else {
      d[f] = rd_col(st + offB[f - TM] + s * 16 * BT * 2);
    }
  };
  auto mf = [&](int m, bf16x8 (&c)[NF]) {
    const int i = m / TN, j = m % TN;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c[TM + j], c[i], acc[i][j], 0, 0, 0);
  };

  // One segment of the contraction: nk k-tiles; DW: rows seg0 .. of the sorted
  // order, whose tokens are in tab.
  const int ld = waveA ? (KIND == kDWGU ? 2 * I : H) : (KIND == kDWGU ? H : I);
  auto run = [&](int nk, int seg0, int segn) {
    auto copy = [&](int kt, int j, int tok) {
      const int ktc = min(kt, nk - 1);  // past the last: copied again, never used
      const bf16* p;
      if constexpr (DW) {
        p = tok < 0 ? zeros : src[j] + (size_t)tok * ld;
      } else {
        if (waveA) {
          p = src[j] + ktc * GK;
        } else if constexpr (KIND == kDU) {
          p = src[j] + (size_t)ktc * GK * I;
        } else {
          p = src[j] + (size_t)ktc * GK * H + (ktc * GK >= I ? up_shift : 0);
        }
      }
      lds_copy16(p, smem + (kt % kStages) * kStageBytes + (wave * LPW + j) * 1024);
    };
    // DW: the row of the source that k row kr of tile kt is, -1 for zeros
    constexpr bool gatherA = KIND == kDWDN;
    auto source_row = [&](int kt, int j) {
      if constexpr (!DW) return 0;
      const int r = min(kt, nk - 1) * GK + kr[j];
      const int tok = tab[r];
      return waveA == gatherA ? tok : (r < segn ? seg0 + r : -1);
    };
    int nx[LPW];
#pragma unroll
    for (int s = 0; s < kStages; ++s)
#pragma unroll
      for (int j = 0; j < LPW; ++j) copy(s, j, source_row(s, j));
    wait_vmem<(kStages - 1) * LPW>();
    block_barrier();
#pragma unroll
    for (int f = 0; f < NF; ++f) rd(smem, 0, f, f0);
    wait_lds();
    __builtin_amdgcn_sched_barrier(0);
    for (int kt = 0; kt < nk; ++kt) {
      const unsigned char* st = smem + (kt % kStages) * kStageBytes;
      const unsigned char* sn = smem + ((kt + 1) % kStages) * kStageBytes;
      // first half: products on f0, reads of the second half's fragments
#pragma unroll
      for (int m = 0; m < NMF; ++m) {
        if (m < NF) rd(st, 1, m, f1);
        mf(m, f0);
        if (m < LPW) nx[m] = source_row(kt + kStages, m);
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_lds();
      // tile kt + 1 has landed for every wave; no wave reads tile kt after this,
      // so its slot takes tile kt + kStages
      wait_vmem<(kStages - 2) * LPW>();
      block_barrier();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < NMF; ++m) {
        if (m < NF) rd(sn, 0, m, f0);
        mf(m, f1);
        if (m >= NMF - LPW) copy(kt + kStages, m - (NMF - LPW), nx[m - (NMF - LPW)]);
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_lds();
    }
    wait_vmem<0>();
    __syncthreads();
  };
  if constexpr (DW) {
    for (int seg0 = row0; seg0 < row1; seg0 += kTab) {
      const int segn = min(kTab, row1 - seg0);
      for (int r = threadIdx.x; r < (segn + GK - 1) / GK * GK; r += 512)
        tab[r] = r < segn ? o.row_tok[seg0 + r] : -1;
      __syncthreads();
      run((segn + GK - 1) / GK, seg0, segn);
    }
  } else {
    run((KIND == kDU ? H : 2 * I) / GK, 0, 0);
  }

  // Epilogue through LDS (the ring's, free now), so that whole rows are read and
  // written in 16-B pieces.
  const int tid = threadIdx.x;
  if constexpr (KIND == kDU) {
    float* stg = reinterpret_cast<float*>(smem);
    const bf16* kept = static_cast<const bf16*>(o.kept);
    bf16* d_gu = static_cast<bf16*>(o.d_gu);
    bf16* hw = static_cast<bf16*>(o.hw);
    for (int pass = 0; pass < BT / kStageRows; ++pass) {
      if (wm == pass) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                               acc[i][j][4 * q + 3]};
              *reinterpret_cast<f32x4*>(stg + (i * 32 + fr) * kF32Pitch + wn * WC + j * 32 +
                                        8 * q + 4 * fq) = v;
            }
      }
      __syncthreads();
      // 32 lanes a row, 8 columns each
#pragma unroll 2
      for (int it = 0; it < kStageRows / 16; ++it) {
        const int rl = it * 16 + tid / 32, c = (tid % 32) * 8;
        const int row = row0 + pass * kStageRows + rl, col = n0 + c;
        float dot = 0.0f;
        if (row < row1 && col < I) {
          const bool live = o.row_tok[row] >= 0;
          const float w = o.ident ? 1.0f : o.topk_w[o.sorted_slots[row]];
          const bf16x8 g = *reinterpret_cast<const bf16x8*>(kept + (size_t)row * 2 * I + col);
          const bf16x8 u = *reinterpret_cast<const bf16x8*>(kept + (size_t)row * 2 * I + I + col);
          bf16x8 og, ou, oh;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float h, dg, du;
            const float v = stg[rl * kF32Pitch + c + j];
            act_grad<true>((float)g[j], (float)u[j], v, h, dg, du);
            dot += v * h;
            og[j] = (bf16)(live ? w * dg : 0.0f);
            ou[j] = (bf16)(live ? w * du : 0.0f);
            oh[j] = (bf16)(live ? w * h : 0.0f);
          }
          if (!live) dot = 0.0f;
          *reinterpret_cast<bf16x8*>(d_gu + (size_t)row * 2 * I + col) = og;
          *reinterpret_cast<bf16x8*>(d_gu + (size_t)row * 2 * I + I + col) = ou;
          *reinterpret_cast<bf16x8*>(hw + (size_t)row * I + col) = oh;
        }
        if (o.part) {
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor(dot, s, kWave);
          if (tid % 32 == 0 && row < row1) o.part[(size_t)nt * o.rows + row] = dot;
        }
      }
      __syncthreads();
    }
  } else {
    // output rows: DX the sorted rows; DW the weight's rows
    auto out_row = [&](int r) -> WT* {
      if constexpr (KIND == kDX) {
        return row0 + r < row1 ? static_cast<WT*>(o.d_xs) + (size_t)(row0 + r) * H : nullptr;
      } else if constexpr (KIND == kDWGU) {
        const int m = m0 + r;
        if (m >= 2 * I) return nullptr;
        return (m < I ? static_cast<WT*>(o.d_gate) + (size_t)m * H
                      : static_cast<WT*>(o.d_up) + (size_t)(m - I) * H) +
               (size_t)e * o.gu_stride;
      } else {
        const int m = m0 + r;
        return m < H ? static_cast<WT*>(o.d_down) + (size_t)e * o.dn_stride + (size_t)m * I
                     : nullptr;
      }
    };
    constexpr bool F32 = std::is_same<WT, float>::value;
    constexpr int SR = F32 ? kStageRows : BT, PITCH = F32 ? kF32Pitch : kBfPitch;
    constexpr int PER = 16 / (int)sizeof(WT), CH = BT / PER;
    WT* stg = reinterpret_cast<WT*>(smem);
    for (int pass = 0; pass < BT / SR; ++pass) {
      if (!F32 || wm == pass) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              typedef WT wx4 __attribute__((ext_vector_type(4)));
              const wx4 v = {from_f32<WT>(acc[i][j][4 * q]), from_f32<WT>(acc[i][j][4 * q + 1]),
                             from_f32<WT>(acc[i][j][4 * q + 2]),
                             from_f32<WT>(acc[i][j][4 * q + 3])};
              const int r = (F32 ? 0 : wm * WR) + i * 32 + fr;
              *reinterpret_cast<wx4*>(stg + r * PITCH + wn * WC + j * 32 + 8 * q + 4 * fq) = v;
            }
      }
      __syncthreads();
      for (int k = tid; k < SR * CH; k += 512) {
        const int r = k / CH, c = (k % CH) * PER;
        WT* dst = out_row(pass * SR + r);
        if (dst && n0 + c < Nout)
          *reinterpret_cast<uint4*>(dst + n0 + c) =
              *reinterpret_cast<const uint4*>(stg + r * PITCH + c);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// fp32 (debug path): 64 x 64 tiles on the vector ALUs
// ---------------------------------------------------------------------------
constexpr int FT = 64, FK = 16;

template <int KIND>
__global__ __launch_bounds__(256) void grad_gemm_f32_kernel(Operands o, int MT, int NT) {
  constexpr bool DW = KIND == kDWGU || KIND == kDWDN;
  __shared__ __align__(16) float As[FK][FT + 4], Bs[FK][FT + 4];
  __shared__ int toks[FT];
  const int H = o.H, I = o.I;
  const int Nout = KIND == kDU || KIND == kDWDN ? I : H;
  const int M = KIND == kDWGU ? 2 * I : H;
  int e = 0, row0, row1, m0 = 0;
  const int nt = blockIdx.x % NT, n0 = nt * FT;
  if constexpr (DW) {
    e = blockIdx.x / (MT * NT);
    m0 = blockIdx.x / NT % MT * FT;
    const bool all = o.ident || o.rows == 0;  // no rows: the offsets may not exist
    row0 = all ? 0 : o.offsets[e];
    row1 = all ? o.rows : o.offsets[e + 1];
  } else if (o.ident) {
    row0 = blockIdx.x / NT * FT;
    row1 = min(row0 + FT, o.rows);
  } else if (!find_row_tile(o.offsets, o.E, FT, blockIdx.x / NT, e, row0, row1)) {
    return;  // uniform over the block
  }
  const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
  const float* d_out = static_cast<const float*>(o.d_out);
  const float* x = static_cast<const float*>(o.x);
  const float* kept = static_cast<const float*>(o.kept);
  float* d_gu = static_cast<float*>(o.d_gu);
  float* hw = static_cast<float*>(o.hw);
  const float* wg = static_cast<const float*>(o.w_gate) + (size_t)e * o.gu_stride;
  const float* wu = static_cast<const float*>(o.w_up) + (size_t)e * o.gu_stride;
  const float* wd = static_cast<const float*>(o.w_down) + (size_t)e * o.dn_stride;
  const int Kd = DW ? row1 - row0 : KIND == kDU ? H : 2 * I;
  if (!DW && tid < FT) toks[tid] = row0 + tid < row1 ? o.row_tok[row0 + tid] : -1;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < Kd; k0 += FK) {
    if (DW && tid < FK) toks[tid] = k0 + tid < Kd ? o.row_tok[row0 + k0 + tid] : -1;
    __syncthreads();
    for (int i = tid; i < FT * FK; i += 256) {
      if constexpr (DW) {
        const int k = i / FT, c = i % FT, r = row0 + k0 + k, tok = toks[k];
        float a = 0.0f, b = 0.0f;
        if (k0 + k < Kd && tok >= 0) {
          if (m0 + c < M)
            a = KIND == kDWGU ? d_gu[(size_t)r * 2 * I + m0 + c] : d_out[(size_t)tok * H + m0 + c];
          if (n0 + c < Nout)
            b = KIND == kDWGU ? x[(size_t)tok * H + n0 + c] : hw[(size_t)r * I + n0 + c];
        }
        As[k][c] = a;
        Bs[k][c] = b;
      } else {
        const int r = i / FK, ka = i % FK;  // contraction lengths are multiples of 32
        float a = 0.0f;
        if (row0 + r < row1) {
          if (KIND == kDU)
            a = toks[r] >= 0 ? d_out[(size_t)toks[r] * H + k0 + ka] : 0.0f;
          else
            a = d_gu[(size_t)(row0 + r) * 2 * I + k0 + ka];
        }
        As[ka][r] = a;
        const int k = i / FT, c = i % FT, kk = k0 + k;
        float b = 0.0f;
        if (n0 + c < Nout) {
          if (KIND == kDU)
            b = wd[(size_t)kk * I + n0 + c];
          else
            b = kk < I ? wg[(size_t)kk * H + n0 + c] : wu[(size_t)(kk - I) * H + n0 + c];
        }
        Bs[k][c] = b;
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < FK; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(&As[k][4 * tr]);
      const float4 b = *reinterpret_cast<const float4*>(&Bs[k][4 * tc]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rl = 4 * tr + i, row = row0 + rl;
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = n0 + 4 * tc + j;
      if (col >= Nout) continue;
      const float v = acc[i][j];
      if constexpr (KIND == kDU) {
        if (row >= row1) continue;
        const bool live = toks[rl] >= 0;
        const float w = o.ident ? 1.0f : o.topk_w[o.sorted_slots[row]];
        float h, dg, du;
        act_grad<false>(kept[(size_t)row * 2 * I + col], kept[(size_t)row * 2 * I + I + col], v, h,
                        dg, du);
        if (live) dot += v * h;
        d_gu[(size_t)row * 2 * I + col] = live ? w * dg : 0.0f;
        d_gu[(size_t)row * 2 * I + I + col] = live ? w * du : 0.0f;
        hw[(size_t)row * I + col] = live ? w * h : 0.0f;
      } else if constexpr (KIND == kDX) {
        if (row < row1) static_cast<float*>(o.d_xs)[(size_t)row * H + col] = v;
      } else {
        const int m = m0 + rl;
        if (m >= M) continue;
        if constexpr (KIND == kDWGU) {
          float* d = m < I ? static_cast<float*>(o.d_gate) + (size_t)m * H
                           : static_cast<float*>(o.d_up) + (size_t)(m - I) * H;
          d[(size_t)e * o.gu_stride + col] = v;
        } else {
          static_cast<float*>(o.d_down)[(size_t)e * o.dn_stride + (size_t)m * I + col] = v;
        }
      }
    }
    if (KIND == kDU && o.part) {
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) dot += __shfl_xor(dot, s, kWave);
      if (tc == 0 && row < row1) o.part[(size_t)nt * o.rows + row] = dot;
    }
  }
}

template <int KIND, typename WT>
hipError_t launch_gemm(const FfnGradArgs& a, const Operands& o, hipStream_t s) {
  constexpr bool DW = KIND == kDWGU || KIND == kDWDN;
  const int N = KIND == kDU || KIND == kDWDN ? a.I : a.H;
  const int M = KIND == kDWGU ? 2 * a.I : a.H;
  const int bt = a.bf16 ? BT : FT;
  const int NT = (N + bt - 1) / bt, MT = (M + bt - 1) / bt;
  const int E = a.ident ? 1 : a.E;
  const int blocks = DW ? E * MT * NT : tile_count_bound(a.ident, a.rows, a.T, a.E, bt) * NT;
  if (blocks == 0) return hipSuccess;
  if (a.bf16) {
    auto kf = grad_gemm_kernel<KIND, WT>;
    static const hipError_t attr = hipFuncSetAttribute(
        reinterpret_cast<const void*>(kf), hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes);
    if (attr != hipSuccess) return attr;
    hipLaunchKernelGGL(kf, dim3(blocks), dim3(512), kLdsBytes, s, o, MT, NT);
  } else {
    hipLaunchKernelGGL(grad_gemm_f32_kernel<KIND>, dim3(blocks), dim3(256), 0, s, o, MT, NT);
  }
  return hipGetLastError();
}

}  // namespace

int ffn_grad_parts(int I, bool bf16) { return bf16 ? (I + BT - 1) / BT : (I + FT - 1) / FT; }

hipError_t launch_ffn_grad(const FfnGradArgs& a, hipStream_t s) {
  Operands o{};
  o.H = a.H; o.I = a.I; o.E = a.ident ? 1 : a.E; o.K = a.K; o.rows = a.rows; o.ident = a.ident;
  o.offsets = a.offsets; o.row_tok = a.ws_row_tok; o.sorted_slots = a.sorted_slots;
  o.topk_w = a.topk_w; o.x = a.x; o.d_out = a.d_out; o.kept = a.kept;
  o.w_gate = a.w_gate; o.w_up = a.w_up; o.w_down = a.w_down;
  o.gu_stride = a.gu_stride; o.dn_stride = a.dn_stride;
  o.d_gu = a.ws_d_gu; o.hw = a.ws_hw; o.part = a.d_topk_w ? a.ws_part : nullptr;
  o.d_xs = a.ident ? a.d_x : a.ws_d_xs;
  o.d_gate = a.d_gate; o.d_up = a.d_up; o.d_down = a.d_down;
  hipError_t e;
  if (a.rows > 0) {
    hipLaunchKernelGGL(rows_kernel, dim3((a.rows + 255) / 256), dim3(256), 0, s, a.rows,
                       (int)a.ident, a.E, a.K, a.offsets, a.sorted_slots, a.mask, a.ws_row_tok,
                       a.ws_slot_row);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = launch_gemm<kDU, bf16>(a, o, s)) != hipSuccess) return e;
    if (a.d_x && (e = launch_gemm<kDX, bf16>(a, o, s)) != hipSuccess) return e;
    if (!a.ident && (a.d_x || a.d_topk_w)) {
      const int parts = ffn_grad_parts(a.I, a.bf16);
      if (a.bf16)
        hipLaunchKernelGGL(combine_grad_kernel<bf16>, dim3(a.T), dim3(256), 0, s, a.T, a.H, a.K,
                           a.E, parts, (long long)a.rows, a.offsets, a.sorted_slots,
                           a.ws_slot_row, static_cast<const bf16*>(a.ws_d_xs), a.ws_part,
                           static_cast<bf16*>(a.d_x), a.d_topk_w);
      else
        hipLaunchKernelGGL(combine_grad_kernel<float>, dim3(a.T), dim3(256), 0, s, a.T, a.H, a.K,
                           a.E, parts, (long long)a.rows, a.offsets, a.sorted_slots,
                           a.ws_slot_row, static_cast<const float*>(a.ws_d_xs), a.ws_part,
                           static_cast<float*>(a.d_x), a.d_topk_w);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  const bool b = a.bf16 && a.wgrad_bf16;
  if (a.d_gate && (e = b ? launch_gemm<kDWGU, bf16>(a, o, s) : launch_gemm<kDWGU, float>(a, o, s)) !=
                      hipSuccess)
    return e;
  if (a.d_down && (e = b ? launch_gemm<kDWDN, bf16>(a, o, s) : launch_gemm<kDWDN, float>(a, o, s)) !=
                      hipSuccess)
    return e;
  return hipSuccess;
}

}  // namespace moe
