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
// Rows are the expert-sorted slots of the dispatch (the dense MLP's: the tokens).  A
// row whose token does not count enters every product as zeros, whatever its token's
// data hold.
//
// Roundings of the bf16 form, all sums being fp32:
//   g, u          as kept by the forward pass: half of the bytes that are kept
//   d_g, d_u, w h operands of the bf16 matrix instructions; two bf16 pieces of each
//                 would double three of the four products
//   d_xs          a slot's part of d_x, in the slots' type: bf16 where the caller takes
//                 bf16 slots, else fp32, at 26B-A4B's 64 / 4096 tokens 577 / 1366 us for
//                 the whole call instead of 549 / 1303
// Error in the root mean square, of its own: d_x 2.3e-3 with fp32 parts, 2.9e-3 with bf16
// ones, the weights' gradients 2.3e-3, d_w 3e-7; rounding the exact value once 1.7e-3.
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr unsigned kNowhere = 0xF0000000u;  // an offset past every buffer here

enum Kind { kDU = 0, kDX = 1, kDWGU = 2, kDWDN = 3 };

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

// d_x[t] = sum over t's slots (k ascending) of their rows of d_xs, in fp32;
// d_topk_w[t, k] = the sum of its row's partial sums (column tiles ascending).
// A block a token, eight rows' loads in flight a thread: 4096 tokens x 8 rows of
// 2816 bf16 in 51 us, 4.1 TB/s (a copy 4.85).
template <typename XT, typename ST>
__global__ __launch_bounds__(256) void combine_grad_kernel(
    int T, int H, int K, int E, int parts, long long part_stride,
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ sorted_slots,
    const int32_t* __restrict__ slot_row, const ST* __restrict__ d_xs,
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
      ST v[8][8];
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int r = k0 + kk < K ? row_of[k0 + kk] : -1;
        if (r >= 0) {
          const uint4* q = reinterpret_cast<const uint4*>(d_xs + (size_t)r * H + c);
#pragma unroll
          for (int i = 0; i < (int)(sizeof(ST) / 2); ++i)
            reinterpret_cast<uint4*>(v[kk])[i] = q[i];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[kk][j] = (ST)0.0f;
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
  int T, H, I, E, K, rows, ident;
  const int32_t* offsets;
  const int32_t* sorted_slots;
  const uint8_t* mask;
  unsigned* row_off;    // row -> its token's byte offset in x and d_out, or kNowhere
  int32_t* slot_row;    // slot -> its row
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

// The token of a row, -1 if it does not count.
__device__ __forceinline__ int token_of(const Operands& o, int row) {
  const int tok = o.ident ? row : o.sorted_slots[row] / o.K;
  return o.mask && !o.mask[tok] ? -1 : tok;
}

// DU writes the tables that the later kernels read, a row tile's by its first block.  A
// slot that the dispatch dropped keeps whatever the workspace held: readers of slot_row
// check that sorted_slots points back.
__device__ __forceinline__ void write_tables(const Operands& o, int row0, int row1,
                                             unsigned row_bytes) {
  for (int r = row0 + threadIdx.x; r < row1; r += blockDim.x) {
    const int tok = token_of(o, r);
    o.row_off[r] = tok < 0 ? kNowhere : (unsigned)tok * row_bytes;
    if (!o.ident) o.slot_row[o.sorted_slots[r]] = r;
  }
}

// ---------------------------------------------------------------------------
// bf16: tiles on v_mfma_f32_32x32x16_bf16
// ---------------------------------------------------------------------------
// Two forms of an operand in LDS, per k-tile of 32:
//  - "row": memory rows run along k (the gathered rows of DU and DX).  64 B a row,
//    16-B chunk c of row r at position c ^ ((r >> 2) & 3); a fragment is one 16-B
//    read.
//  - "col": memory rows are the k index (weights of DU and DX, both operands of
//    the weight gradients).  32 rows as wide as the tile, 32-B piece p of row k at
//    position p ^ (2 (k & 3)), p ^ (k & 3) in rows of 64 columns; a fragment is two
//    transposing 8-B reads
//    (ds_read_b64_tr_b16: each group of 16 lanes reads four k of 16 columns, lane
//    i gets column i).  The four k of a group lie in four pieces and the next
//    group's four in the other four of the same 256 B: no bank twice.
// Both come in by direct global -> LDS copies into a ring of stages.  The B
// columns are the instruction's first operand, so a lane's results are runs of
// four consecutive columns of one row.
constexpr int GK = 32;

__device__ __forceinline__ int rswz(int r, int c) { return c ^ ((r >> 2) & 3); }
__device__ __forceinline__ int cswz(int k, int p, int width) {
  return p ^ (width >= 128 ? (k & 3) << 1 : k & 3);
}

// BM x BN tile, WM x WN waves, ST stages, blocks that share a CU.
template <int BM_, int BN_, int WM_, int WN_, int ST_, int BLOCKS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_, NW = WM * WN;
  static constexpr int BLOCKS = BLOCKS_, WAVES_EU = (BLOCKS_ * NW + 3) / 4;  // waves a SIMD
  static constexpr int A_BYTES = BM * GK * 2, B_BYTES = BN * GK * 2, STAGE = A_BYTES + B_BYTES;
  static constexpr int RING = ST * STAGE;
  static constexpr int WR = BM / WM, WC = BN / WN, TM = WR / 32, TN = WC / 32;
  // LDS of a block that stages its results over the ring: WR rows of fp32 or BM of bf16
  static constexpr int F32_PITCH = BN + 4, BF_PITCH = BN + 8;
  static constexpr int STAGED = WR * F32_PITCH * 4 > BM * BF_PITCH * 2 ? WR * F32_PITCH * 4
                                                                       : BM * BF_PITCH * 2;
  // (with the contraction split over KS groups, the fp32 of all of them)
  template <int KS>
  static constexpr int rows_lds() {
    const int staged = KS > 1 ? KS * BM * F32_PITCH * 4 : STAGED;
    return KS * RING > staged ? KS * RING : staged;
  }
  // LDS through which a wave's results leave: 32 rows of SJ 32-column sub-tiles
  static constexpr int SJ = BLOCKS * (RING + NW * 4096) <= 160 * 1024 ? 2 : 1;
  static constexpr int WAVE_STAGING = SJ * 2048;
  static constexpr int NF = TM + TN, NMF = TM * TN;  // fragments, products a half k-tile
  static constexpr int CA = A_BYTES / 1024 / NW, CB = B_BYTES / 1024 / NW;  // copies a wave
  static constexpr int LPW = CA + CB;
  // col form: lanes a k row, k rows a copy, copies after which the swizzle repeats
  static constexpr int LA = BM / 8, LB = BN / 8, SA = 64 / LA, SB = 64 / LB;
  static constexpr int PA = SA >= 4 ? 1 : (4 / SA < CA ? 4 / SA : CA);
  static constexpr int PB = SB >= 4 ? 1 : (4 / SB < CB ? 4 / SB : CB);
  static_assert(CA * NW * 1024 == A_BYTES && CB * NW * 1024 == B_BYTES, "whole copies");
  static_assert(BN >= 64, "the col form's swizzle needs 4 pieces a row");
  static_assert(ST >= 2, "waits");
};

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(4))) const int const_int;

// LDS offset of a shared array.
__device__ __forceinline__ unsigned lds_offset(unsigned char* p) {
#if defined(__HIP_DEVICE_COMPILE__)
  return (unsigned)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)p;
#else
  return (unsigned)(uintptr_t)p;
#endif
}

// A fragment of the row form at LDS offset a; of the col form, its k rows 0..3 at a
// and 4..7 `step` bytes on.
__device__ __forceinline__ bf16x8 frag_row(unsigned a) {
#if defined(__HIP_DEVICE_COMPILE__)
  return *(lds_bf16x8*)a;
#else
  return bf16x8{};
#endif
}
__device__ __forceinline__ bf16x8 frag_col(unsigned a, int step) {
  union {
    s16x4 h[2];
    bf16x8 v;
  } u = {};
#if defined(__HIP_DEVICE_COMPILE__)
  u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
  u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + step));
#endif
  return u.v;
}

// Descriptor of `bytes` bytes at p: loads past them give zeros, stores past them
// are dropped.  Uniform over the wave.
__device__ __forceinline__ i32x4 buffer_of(const void* p, unsigned bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  i32x4 d;
  d[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  d[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu));
  d[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  d[3] = 0x00020000;
  return d;
}

// Copies and stores through descriptors, in inline asm for the reason given at
// lds_copy16 and so that the waits below count them exactly.  The compiler does not
// see these instructions, so their wait states are here: five after a vector
// instruction that wrote a scalar register they read (readfirstlane), two before a
// vector instruction that overwrites a store's data.
__device__ __forceinline__ void buffer_copy16(i32x4 buf, unsigned off, unsigned lds) {
  const unsigned m0 = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(buf), "s"(m0)
               : "memory", "m0");
}
// `at`: bytes that all lanes add
__device__ __forceinline__ void buffer_copy16(i32x4 buf, unsigned off, unsigned at,
                                              unsigned lds) {
  const unsigned m0 = __builtin_amdgcn_readfirstlane(lds);
  const unsigned so = __builtin_amdgcn_readfirstlane(at);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds"
               :
               : "v"(off), "s"(buf), "s"(m0), "s"(so)
               : "memory", "m0");
}
template <bool ONCE>
__device__ __forceinline__ void global_copy16(const void* base, unsigned off, unsigned lds) {
  const unsigned m0 = __builtin_amdgcn_readfirstlane(lds);
  if constexpr (ONCE)  // leaves the caches first
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1 nt"
                 :
                 : "v"(off), "s"(base), "s"(m0)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(base), "s"(m0)
                 : "memory", "m0");
}
template <bool PAST>
__device__ __forceinline__ void buffer_store16(i32x4 buf, unsigned off, i32x4 v) {
  if constexpr (PAST)  // past the caches
    asm volatile("s_nop 4\n\tbuffer_store_dwordx4 %0, %1, %2, 0 offen nt\n\ts_nop 1"
                 :
                 : "v"(v), "v"(off), "s"(buf)
                 : "memory");
  else
    asm volatile("s_nop 4\n\tbuffer_store_dwordx4 %0, %1, %2, 0 offen\n\ts_nop 1"
                 :
                 : "v"(v), "v"(off), "s"(buf)
                 : "memory");
}

// Fragment offsets of a wave within a stage.
template <typename TL, bool ROW_A>
struct FragOffsets {
  unsigned a[ROW_A ? 1 : TL::TM], b[TL::TN];
  __device__ __forceinline__ FragOffsets(int lane, int wm, int wn) {
    // row form: lane -> row lane % 32, chunk lane / 32 (+ 2 for the second half)
    const int fr = lane % 32, fq = lane / 32;
    // col form: k = 8 fq + (lane % 16) / 4, columns c .. c + 3 of the lane's address
    const int tk = 8 * fq + (lane % 16) / 4, tc = 16 * ((lane / 16) % 2) + 4 * (lane % 4);
    auto col = [&](int c, int width) {
      c += tc;
      return (unsigned)(tk * width * 2 + cswz(tk, c / 16, width) * 32 + (c % 16) * 2);
    };
    if constexpr (ROW_A) {
      const int r = wm * TL::WR + fr;  // 32 rows on, the swizzle is the same
      a[0] = r * 64 + rswz(r, fq) * 16;
    } else {
#pragma unroll
      for (int i = 0; i < TL::TM; ++i) a[i] = col(wm * TL::WR + i * 32, TL::BM);
    }
#pragma unroll
    for (int j = 0; j < TL::TN; ++j) b[j] = TL::A_BYTES + col(wn * TL::WC + j * 32, TL::BN);
  }
  // fragment f (A's TM, then B's TN) of half s of the stage at offset st
  __device__ __forceinline__ bf16x8 read(unsigned st, int s, int f) const {
    if (f >= TL::TM)
      return frag_col(b[f - TL::TM] + st + s * 16 * TL::BN * 2, 4 * TL::BN * 2);
    if constexpr (ROW_A) return frag_row((a[0] ^ (s * 32)) + st + f * 32 * 64);
    else return frag_col(a[f] + st + s * 16 * TL::BM * 2, 4 * TL::BM * 2);
  }
};

template <typename TL>
__device__ __forceinline__ void clear(f32x16 (&acc)[TL::TM][TL::TN]) {
#pragma unroll
  for (int i = 0; i < TL::TM; ++i)
#pragma unroll
    for (int j = 0; j < TL::TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
}

// DU and DX: a block takes one row tile of one expert and one column tile.  Its KS
// groups of waves split the contraction, each with a ring of its own; their sums meet
// in LDS, always in the same order.
// The experts' 128 x 256 tiles at 4096 tokens (256 rows an expert on average, so three
// row tiles with their last ones half empty, neighbours on one XCD for their weights):
// DU 284 us, 457 TFLOP/s, DX 391 us, 664 TFLOP/s, the matrix units busy for 0.27 and
// 0.41 of the time; a wave's LDS reads take nearly as long as its products, and the
// weights (1.5 GB for the two) come from memory once.  (Kernel times here and below are
// of a trace of the call alone; they differ by up to 5 % from card to card, and those
// compared with each other are of one card.)  DU's contraction of 88 k-tiles
// ends in an epilogue that reads the kept projections and writes 1.5 times as much; the
// second block of the CU multiplies meanwhile.  At 64 tokens the weights bound both:
// 90 and 128 us, 4.8 and 6.8 TB/s.
// ONCE: the weights' copies do not stay in the caches.
template <int KIND, typename WT, typename TL, int KS, bool ONCE>
__device__ __forceinline__ void rows_block(const Operands& o, int NT, int block,
                                           unsigned char* smem) {
  constexpr int BM = TL::BM, BN = TL::BN, NW = TL::NW, ST = TL::ST, WN = TL::WN;
  constexpr int TM = TL::TM, TN = TL::TN, NF = TL::NF, NMF = TL::NMF, WR = TL::WR, WC = TL::WC;
  constexpr int CA = TL::CA, LPW = TL::LPW;
  static_assert(KS == 1 || NW == 1, "groups of several waves would wait for each other");

  const int H = o.H, I = o.I;
  const int Nout = KIND == kDU ? I : H;
  int e = 0, row0, row1, nt;
  {
    RowTileScan sc;
    int R;
    if (o.ident) {
      R = (o.rows + BM - 1) / BM;
    } else {
      row_tile_scan(o.offsets, o.E, BM, sc);
      R = sc.total;
    }
    const int item = xcd_item(block, R * NT);
    if (item < 0) return;  // uniform over the block
    if (o.ident) {
      nt = item % NT;
      row0 = item / NT * BM;
      row1 = min(row0 + BM, o.rows);
    } else {
      weight_major_item(sc, o.offsets, BM, item, NT, e, row0, row1, nt);
    }
  }
  e = __builtin_amdgcn_readfirstlane(e);
  nt = __builtin_amdgcn_readfirstlane(nt);
  row0 = __builtin_amdgcn_readfirstlane(row0);
  row1 = __builtin_amdgcn_readfirstlane(row1);
  const int lane = lane_id(), block_wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int grp = block_wave / NW, wave = block_wave % NW;
  const unsigned base = lds_offset(smem) + grp * TL::RING;
  const int wm = wave / WN, wn = wave % WN, fr = lane % 32, fq = lane / 32;
  const int n0 = nt * BN;

  if (KIND == kDU && nt == 0) write_tables(o, row0, row1, 2u * (unsigned)H);

  // This lane's copies of a k-tile, CA of A and CB of B: byte offsets from bases
  // that all lanes share.  A row past the tile and a token that does not count lie
  // outside A's descriptor: zeros, and no traffic.
  unsigned off[LPW], atA = 0;
  const bf16 *pB, *pU = nullptr;
  i32x4 bufA;
  if constexpr (KIND == kDU) {
    bufA = buffer_of(o.d_out, (unsigned)o.T * 2u * (unsigned)H);
    pB = static_cast<const bf16*>(o.w_down) + (size_t)e * o.dn_stride;
  } else {
    bufA = buffer_of(static_cast<const bf16*>(o.d_gu) + (size_t)row0 * 2 * I,
                     (unsigned)(row1 - row0) * 4u * (unsigned)I);
    pB = static_cast<const bf16*>(o.w_gate) + (size_t)e * o.gu_stride;
    pU = static_cast<const bf16*>(o.w_up) + (size_t)e * o.gu_stride;
  }
#pragma unroll
  for (int j = 0; j < LPW; ++j) {
    if (j < CA) {
      const int r = 16 * (wave * CA + j) + lane / 4;
      if constexpr (KIND == kDU) {
        const int tok = row0 + r < row1 ? token_of(o, row0 + r) : -1;
        off[j] = tok < 0 ? kNowhere : (unsigned)tok * (unsigned)(2 * H) + rswz(r, lane % 4) * 16;
      } else {
        off[j] = row0 + r < row1 ? (unsigned)r * (unsigned)(4 * I) + rswz(r, lane % 4) * 16
                                 : kNowhere;
      }
    } else {
      const int k = TL::SB * (wave * TL::CB + j - CA) + lane / TL::LB;
      const int c = n0 + cswz(k, lane % TL::LB / 2, BN) * 16 + (lane & 1) * 8;
      off[j] = ((unsigned)k * (unsigned)Nout + (unsigned)(c < Nout ? c : 0)) * 2u;
    }
  }
  // this group's k-tiles
  const int nk_all = (KIND == kDU ? H : 2 * I) / GK, first = grp * nk_all / KS;
  const int nk = (grp + 1) * nk_all / KS - first;
  // atA, pB: the k-tile that is being copied; `turn` k-tiles before pB goes on to the
  // up rows
  int turn = KIND == kDX ? I / GK - first : -1;
  atA += first * GK * 2;
  if (KIND == kDX && turn <= 0) pB = pU + (size_t)(-turn) * GK * Nout;
  else pB += (size_t)first * GK * Nout;
  const unsigned ldsA = base + wave * CA * 1024, ldsB = base + TL::A_BYTES + wave * TL::CB * 1024;
  auto copy = [&](int j, unsigned st) {
    if (j < CA) buffer_copy16(bufA, off[j], atA, ldsA + st + j * 1024);
    else global_copy16<ONCE>(pB, off[j], ldsB + st + (j - CA) * 1024);
  };
  auto copied = [&]() {
    atA += GK * 2;
    pB += (size_t)GK * Nout;
    if (KIND == kDX && --turn == 0) pB = pU;
  };
  // 32-row sub-tiles of this wave that hold rows
  int nv;
  {
    const int left = row1 - row0 - wm * WR;
    nv = left <= 0 ? 0 : min(TM, (left + 31) / 32);
  }
  const FragOffsets<TL, true> fo(lane, wm, wn);
  f32x16 acc[TM][TN];
  clear<TL>(acc);

  // a group of one wave has its ring for itself and waits for nobody
  auto group_barrier = [&]() {
    if constexpr (NW > 1) block_barrier();
    else asm volatile("" ::: "memory");
  };

  auto run = [&](auto nv_tag) {
    constexpr int NV = decltype(nv_tag)::value;  // sub-tiles of rows to multiply
    bf16x8 f0[NF], f1[NF];
    auto rd = [&](unsigned st, int s, int f, bf16x8 (&d)[NF]) {
      if (NV > 0 && (f >= TM || f < NV)) d[f] = fo.read(base + st, s, f);
    };
    auto mf = [&](int m, bf16x8 (&c)[NF]) {
      const int i = m / TN, j = m % TN;
      if (i < NV)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c[TM + j], c[i], acc[i][j], 0, 0, 0);
    };
    // waits until all but the last `tiles` tiles' copies have landed
    auto wait_tiles = [&](int tiles) {
      if (tiles >= ST - 1) wait_vmem<(ST - 1) * LPW>();
      else if (tiles == ST - 2) wait_vmem<(ST - 2) * LPW>();
      else if (ST > 3 && tiles == 1) wait_vmem<LPW>();
      else wait_vmem<0>();
    };
    // The copies of tile kt + ST go to tile kt's slot: the first P1 of them in the
    // second half of tile kt, when no wave reads it any more, the others in the first
    // half of tile kt + 1, so that the copy path is never idle for half of the time
    // (with two stages all at once: they have a tile less to arrive).
    constexpr int P1 = ST == 2 ? LPW : LPW / 2, P2 = LPW - P1;
#pragma unroll
    for (int s = 0; s < ST; ++s)
      if (s < nk) {
#pragma unroll
        for (int j = 0; j < LPW; ++j)
          if (s < ST - 1 || j < P1) copy(j, s * TL::STAGE);
        if (s < ST - 1) copied();
      }
    if (nk >= ST) wait_vmem<(ST - 2) * LPW>();
    else wait_tiles(nk - 1);
    group_barrier();
#pragma unroll
    for (int f = 0; f < NF; ++f) rd(0, 0, f, f0);
    wait_lds();
    __builtin_amdgcn_sched_barrier(0);
    unsigned cur = 0, prv = TL::RING - TL::STAGE;
    auto tile = [&](int kt, auto first_tag, auto second_tag) {
      constexpr bool FIRST = decltype(first_tag)::value;    // tile kt - 1 + ST exists
      constexpr bool SECOND = decltype(second_tag)::value;  // tile kt + ST exists
      const unsigned nxt = cur + TL::STAGE == TL::RING ? 0 : cur + TL::STAGE;
      // first half: products on f0, reads of the second half's fragments
#pragma unroll
      for (int m = 0; m < NMF; ++m) {
#pragma unroll
        for (int f = m * NF / NMF; f < (m + 1) * NF / NMF; ++f) rd(cur, 1, f, f1);
        mf(m, f0);
        if constexpr (FIRST) {
#pragma unroll
          for (int j = m * P2 / NMF; j < (m + 1) * P2 / NMF; ++j) copy(P1 + j, prv);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (FIRST) copied();
      wait_lds();
      // tile kt + 1 has landed for every wave; no wave reads tile kt after this
      if constexpr (FIRST) wait_vmem<(ST - 2) * LPW>();
      else wait_tiles(nk - 2 - kt);
      group_barrier();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < NMF; ++m) {
#pragma unroll
        for (int f = m * NF / NMF; f < (m + 1) * NF / NMF; ++f) rd(nxt, 0, f, f0);
        mf(m, f1);
        if constexpr (SECOND) {
#pragma unroll
          for (int j = m * P1 / NMF; j < (m + 1) * P1 / NMF; ++j) copy(j, cur);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_lds();
      prv = cur;
      cur = nxt;
    };
    int kt = 0;
    for (; kt + ST < nk; ++kt) tile(kt, std::true_type{}, std::true_type{});
    if (kt + ST == nk) tile(kt++, std::true_type{}, std::false_type{});
    for (; kt < nk; ++kt) tile(kt, std::false_type{}, std::false_type{});
    __syncthreads();
  };
  static_assert(TM == 2, "the cases below");
  if (nv == 2) run(std::integral_constant<int, 2>{});
  else if (nv == 1) run(std::integral_constant<int, 1>{});
  else run(std::integral_constant<int, 0>{});

  // Epilogue through LDS (the rings', free now), so that whole rows are read and
  // written in 16-B pieces; the groups' sums meet there, always in the same order.
  const int tid = threadIdx.x;
  constexpr int F32_PITCH = TL::F32_PITCH, BF_PITCH = TL::BF_PITCH;
  constexpr bool F32 = KIND == kDU || std::is_same<WT, float>::value || KS > 1;
  if constexpr (F32) {
    float* stg = reinterpret_cast<float*>(smem);
    const bf16* kept = static_cast<const bf16*>(o.kept);
    bf16* d_gu = static_cast<bf16*>(o.d_gu);
    bf16* hw = static_cast<bf16*>(o.hw);
    constexpr int LPR = BN / 8, RPI = 64 * NW * KS / LPR;  // lanes a row, rows an iteration
    static_assert(LPR <= kWave && WR % RPI == 0, "rows of the epilogue");
    for (int pass = 0; pass < TL::WM; ++pass) {
      if (wm == pass) {
        float* to = stg + (grp * BM + fr) * F32_PITCH + wn * WC + 4 * fq;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                               acc[i][j][4 * q + 3]};
              *reinterpret_cast<f32x4*>(to + i * 32 * F32_PITCH + j * 32 + 8 * q) = v;
            }
      }
      __syncthreads();
#pragma unroll 2
      for (int it = 0; it < WR / RPI; ++it) {
        const int rl = it * RPI + tid / LPR, c = (tid % LPR) * 8;
        const int row = row0 + pass * WR + rl, col = n0 + c;
        f32x4 va[2];  // the row's eight columns
        auto sums = [&]() {
          const f32x4* from = reinterpret_cast<const f32x4*>(stg + rl * F32_PITCH + c);
          va[0] = from[0];
          va[1] = from[1];
#pragma unroll
          for (int g = 1; g < KS; ++g) {
            va[0] += from[g * (BM * F32_PITCH / 4)];
            va[1] += from[g * (BM * F32_PITCH / 4) + 1];
          }
        };
        if constexpr (KIND == kDX) {
          if (row < row1 && col < Nout) {
            sums();
            WT* d = static_cast<WT*>(o.d_xs) + (size_t)row * H + col;
            if constexpr (std::is_same<WT, float>::value) {
              *reinterpret_cast<f32x4*>(d) = va[0];
              *reinterpret_cast<f32x4*>(d + 4) = va[1];
            } else {
              bf16x8 v;  // d_x itself, or a part of it in the slots' type
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = (bf16)va[j / 4][j % 4];
              *reinterpret_cast<bf16x8*>(d) = v;
            }
          }
        } else {
          float dot = 0.0f;
          if (row < row1 && col < I) {
            const bool live = token_of(o, row) >= 0;
            const float w = o.ident ? 1.0f : o.topk_w[o.sorted_slots[row]];
            const bf16x8 g = *reinterpret_cast<const bf16x8*>(kept + (size_t)row * 2 * I + col);
            const bf16x8 u =
                *reinterpret_cast<const bf16x8*>(kept + (size_t)row * 2 * I + I + col);
            bf16x8 og, ou, oh;
            sums();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float h, dg, du;
              const float v = va[j / 4][j % 4];
              act_grad<true>((float)g[j], (float)u[j], v, h, dg, du);
              dot += v * h;
              // rounded once, from fp32: operands of DX, DWGU and DWDN
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
            for (int s = LPR / 2; s > 0; s >>= 1) dot += __shfl_xor(dot, s, kWave);
            if (tid % LPR == 0 && row < row1) o.part[(size_t)nt * o.rows + row] = dot;
          }
        }
      }
      __syncthreads();
    }
  } else {
    bf16* stg = reinterpret_cast<bf16*>(smem);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // d_x itself, or a part of it in the slots' type
          const bf16x4 v = {(bf16)acc[i][j][4 * q], (bf16)acc[i][j][4 * q + 1],
                            (bf16)acc[i][j][4 * q + 2], (bf16)acc[i][j][4 * q + 3]};
          *reinterpret_cast<bf16x4*>(stg + (wm * WR + i * 32 + fr) * BF_PITCH + wn * WC + j * 32 +
                                     8 * q + 4 * fq) = v;
        }
    __syncthreads();
    constexpr int CH = BN / 8;
#pragma unroll 4
    for (int k = tid; k < BM * CH; k += 64 * NW * KS) {
      const int r = k / CH, c = (k % CH) * 8;
      if (row0 + r < row1 && n0 + c < Nout)
        *reinterpret_cast<uint4*>(static_cast<bf16*>(o.d_xs) + (size_t)(row0 + r) * H + n0 + c) =
            *reinterpret_cast<const uint4*>(stg + r * BF_PITCH + c);
    }
  }
}

template <int KIND, typename WT, typename TL, int KS, bool ONCE>
__global__ __launch_bounds__(64 * TL::NW * KS, (TL::BLOCKS * TL::NW * KS + 3) / 4) void
grad_rows_kernel(Operands o, int NT) {
  extern __shared__ __align__(16) unsigned char smem[];
  rows_block<KIND, WT, TL, KS, ONCE>(o, NT, blockIdx.x, smem);
}

// First tile of the weights' gradients (tpe an expert) that XCD x takes, x = 8: all
// of them.  A tile costs its k-tiles and kTileEnds more for its ends; XCD x starts at
// the first tile that x / 8 of the whole cost lies before.
constexpr int kTileEnds = 3;
__device__ __forceinline__ int first_tile(const Operands& o, int tpe, int x) {
  if (o.ident || o.rows == 0) return (int)((long long)o.E * tpe * x / 8);
  const int lane = lane_id(), per = (o.E + kWave - 1) / kWave;  // experts a lane, <= 4
  int cost[4], mine = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = lane * per + j;
    cost[j] = j < per && e < o.E ? (o.offsets[e + 1] - o.offsets[e] + GK - 1) / GK + kTileEnds : 0;
    mine += cost[j];
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int t = __shfl_up(upto, d, kWave);
    if (lane >= d) upto += t;
  }
  const int total = __shfl(upto, kWave - 1, kWave);
  // in units of an expert's tiles: cost before the target, of E experts at most
  const long long target = (long long)total * x * tpe / 8;
  long long before = (long long)(upto - mine) * tpe;
  int first = 0;  // tiles of this lane's experts that lie before the target
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (cost[j] > 0 && before < target) {
      const long long n = (target - before + cost[j] - 1) / cost[j];
      first += n < tpe ? (int)n : tpe;
    }
    before += (long long)cost[j] * tpe;
  }
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) first += __shfl_xor(first, d, kWave);
  return __builtin_amdgcn_readfirstlane(first);
}

// DWGU and DWDN: the gradients of the weights.  The contraction runs over an
// expert's rows, some 256 of them: 8 k-tiles for a tile that writes 64 KB.  So a
// block goes through many tiles as ONE stream of k-tiles: the copies run ST
// k-tiles ahead of the products, across the tiles' ends, and the results leave from
// the registers (through 4 KB of LDS a wave) while the next tile's copies are under
// way.  (One tile a block, its ring filled and drained each time, ran at 427
// TFLOP/s at 4096 tokens, the matrix unit busy for 0.24 of the time.)
// An operand is "regular" (rows of the sorted order: d_gu, w h) or "gathered" (by
// the rows' tokens: x, d_out).  Both are copied through descriptors, whose range
// check gives zeros for rows past the expert's and for tokens that do not count.
// PAST: the results go past the caches, where they would be written back while later
// kernels read (gradients of 1.5 GB, the next call's DU at 64 / 4096 tokens 90 / 284 us
// against 93 / 298).
template <int KIND, typename WT, typename TL, bool PAST>
__device__ __forceinline__ void weights_block(const Operands& o, int MT, int NT, int block,
                                              int blocks, unsigned char* smem) {
  constexpr int ST = TL::ST, WN = TL::WN, NW = TL::NW;
  constexpr int TM = TL::TM, TN = TL::TN, NF = TL::NF, NMF = TL::NMF, WR = TL::WR, WC = TL::WC;
  constexpr int CA = TL::CA, CB = TL::CB, LPW = TL::LPW;
  constexpr bool GB = KIND == kDWGU;  // B is the gathered operand, else A
  constexpr bool F32 = std::is_same<WT, float>::value;
  constexpr int NS = TM * TN * (F32 ? 4 : 2);  // stores of a tile's results a wave
  constexpr int KW = GK / NW;         // k rows that a wave copies of each operand
  static_assert(TL::SA * CA == KW && TL::SB * CB == KW && (KW & (KW - 1)) == 0, "k rows a wave");
  const unsigned base = lds_offset(smem);
  const int H = o.H, I = o.I;
  const int M = KIND == kDWGU ? 2 * I : H, N = KIND == kDWGU ? H : I;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN, fr = lane % 32, fq = lane / 32;

  // This block's tiles: every nb-th of its XCD's range (neighbours share operands).
  // The ranges split the tiles by their k-tiles, not by their number: experts differ
  // by more than ten in their rows, sixteen of them together by a fifth.
  const int nb = blocks / 8;
  const int end = first_tile(o, MT * NT, block % 8 + 1);
  int c_it = first_tile(o, MT * NT, block % 8) + block / 8;

  const_int* offsets = (const_int*)o.offsets;
  const_int* row_off_tab = (const_int*)o.row_off;
  auto rows_of = [&](int it, int& row0, int& n) {
    if (o.ident || o.rows == 0) {  // no rows: the offsets may not exist
      row0 = 0;
      n = o.rows;
    } else {
      const int e = it / (MT * NT);
      row0 = offsets[e];
      n = offsets[e + 1] - row0;
    }
  };

  // Copies: the k rows of a wave are KW wave .. KW wave + KW - 1 of a k-tile, in CA
  // (CB) copies of SA (SB) rows.  Lane offsets within a k-tile, from the tile's first
  // column: whole ones for the regular operand, the column's part for the gathered.
  constexpr int CR = GB ? CA : CB, CG = GB ? CB : CA;      // copies
  constexpr int SR = GB ? TL::SA : TL::SB, SG = GB ? TL::SB : TL::SA;
  constexpr int LR = GB ? TL::LA : TL::LB, LG = GB ? TL::LB : TL::LA;
  constexpr int PG = GB ? TL::PB : TL::PA;
  const char* Rp = static_cast<const char*>(GB ? o.d_gu : o.hw);
  const char* Gp = static_cast<const char*>(GB ? o.x : o.d_out);
  const unsigned ldr = 2u * (unsigned)(GB ? 2 * I : I), ldg = 2u * (unsigned)H;  // bytes
  auto piece = [&](int k, int lpr) {
    return (unsigned)(cswz(k, lane % lpr / 2, lpr * 8) * 32 + (lane & 1) * 16);
  };
  unsigned offR[CR], colG[PG];
#pragma unroll
  for (int j = 0; j < CR; ++j) {
    const int k = KW * wave + SR * j + lane / LR;
    offR[j] = (unsigned)k * ldr + piece(k, LR);
  }
#pragma unroll
  for (int j = 0; j < PG; ++j) colG[j] = piece(KW * wave + SG * j + lane / LG, LG);
  const unsigned ldsR = base + (GB ? 0 : TL::A_BYTES) + wave * CR * 1024;
  const unsigned ldsG = base + (GB ? TL::A_BYTES : 0) + wave * CG * 1024;

  // The producer: the tile whose k-tiles are being copied.
  int p_it = c_it, p_row0 = 0, p_n = 0, p_k = 0;
  unsigned p_colR = 0;         // bytes of the tile's first column
  const char* p_R = Rp;        // the regular operand's k-tile
  i32x4 bufR = buffer_of(Rp, 0), bufG = buffer_of(Gp, 0);
  auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  int q_it = c_it, q_row0 = 0, q_n = 0;  // the tile after it, fetched ahead
  if (q_it < end) rows_of(q_it, q_row0, q_n);
  auto p_open = [&]() {  // to the next tile with rows
    do {
      p_it = q_it;
      p_row0 = uni(q_row0);
      p_n = uni(q_n);
      q_it += nb;
      if (q_it < end) rows_of(q_it, q_row0, q_n);
    } while (p_it < end && p_n == 0);
    if (p_it < end) {
      const int mt = p_it / NT % MT, nt = p_it % NT;
      p_colR = (unsigned)uni(2 * (GB ? mt * TL::BM : nt * TL::BN));
      const unsigned cg = (unsigned)uni(2 * (GB ? nt * TL::BN : mt * TL::BM));
      p_R = Rp + (size_t)p_row0 * ldr + p_colR;
      bufG = buffer_of(Gp + cg, (unsigned)o.T * ldg - cg);
      p_k = 0;
    }
  };
  unsigned row_off[KW];  // gathered: byte offsets of this wave's k rows
  auto p_rows = [&]() {
    const int left = p_n - p_k;
    bufR = buffer_of(p_R, (unsigned)min(GK, left) * ldr - p_colR);
    const const_int* t = row_off_tab + p_row0 + p_k + KW * wave;  // 32 entries past the last exist
#pragma unroll
    for (int i = 0; i < KW; ++i) row_off[i] = (unsigned)t[i];
    if (left < GK) {  // the rows past the expert's: another's, or none
#pragma unroll
      for (int i = 0; i < KW; ++i)
        if (KW * wave + i >= left) row_off[i] = kNowhere;
    }
  };
  auto p_copy = [&](int j, unsigned st) {  // copy j of a k-tile: the regular ones first
    if (j < CR) {
      buffer_copy16(bufR, offR[j], ldsR + st + j * 1024);
    } else {
      const int g = j - CR;
      unsigned at;
      if constexpr (SG == 2) {
        at = lane < 32 ? row_off[(2 * g) & (KW - 1)] : row_off[(2 * g + 1) & (KW - 1)];
      } else {
        const unsigned lo =
            lane & 16 ? row_off[(4 * g + 1) & (KW - 1)] : row_off[(4 * g) & (KW - 1)];
        const unsigned hi =
            lane & 16 ? row_off[(4 * g + 3) & (KW - 1)] : row_off[(4 * g + 2) & (KW - 1)];
        at = lane & 32 ? hi : lo;
      }
      buffer_copy16(bufG, at + colG[(g < 0 ? 0 : g) % PG], ldsG + st + g * 1024);
    }
  };
  auto p_next = [&]() {
    p_k += GK;
    p_R += (size_t)GK * ldr;
    if (p_k >= p_n) p_open();
  };
  static_assert(SG == 2 || SG == 4, "rows of a gathered copy");

  const FragOffsets<TL, false> fo(lane, wm, wn);
  f32x16 acc[TM][TN];
  bf16x8 f0[NF], f1[NF];
  unsigned cur = 0, prv = TL::RING - TL::STAGE;
  // As in DU and DX, the copies of a k-tile are issued in two parts: the regular
  // operand's in the second half of the k-tile ST before it, while its tokens are on
  // their way, the gathered one's in the first half of the next; `open`: the
  // producer's k-tile has its first part under way.
  constexpr int P1 = CR, P2 = CG;
  bool open = false;
  p_open();
  {  // the stream's first ST k-tiles
#pragma unroll
    for (int s = 0; s < ST; ++s)
      if (p_it < end) {
        p_rows();
#pragma unroll
        for (int j = 0; j < LPW; ++j)
          if (s < ST - 1 || j < P1) p_copy(j, s * TL::STAGE);
        if (s < ST - 1) p_next();
        else open = true;
      }
    wait_vmem<0>();
    block_barrier();
#pragma unroll
    for (int f = 0; f < NF; ++f) f0[f] = fo.read(base, 0, f);
    wait_lds();
  }
  // k-tiles since the last stores: for ST - 2 of them the copies waited for are
  // older than those stores, which may then be outstanding too
  int since = ST;
  for (; c_it < end; c_it += nb) {
    int row0, n;
    rows_of(c_it, row0, n);
    clear<TL>(acc);
    auto tile = [&](auto steady_tag) {
      // the producer's k-tile has its first part under way and the tile has another
      constexpr bool STEADY = decltype(steady_tag)::value;
      const unsigned nxt = cur + TL::STAGE == TL::RING ? 0 : cur + TL::STAGE;
      const bool was_open = STEADY || open;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < NMF; ++m) {
#pragma unroll
        for (int f = m * NF / NMF; f < (m + 1) * NF / NMF; ++f) f1[f] = fo.read(base + cur, 1, f);
        acc[m / TN][m % TN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            f0[TM + m % TN], f0[m / TN], acc[m / TN][m % TN], 0, 0, 0);
        if (was_open) {
#pragma unroll
          for (int j = m * P2 / NMF; j < (m + 1) * P2 / NMF; ++j) p_copy(P1 + j, prv);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (STEADY) {
        p_k += GK;
        p_R += (size_t)GK * ldr;
      } else if (was_open) {
        p_next();
        open = p_it < end;
      }
      wait_lds();
      // the next k-tile has landed for every wave; no wave reads this one after the
      // barrier, so its slot takes the one ST further on
      if (!was_open) wait_vmem<0>();
      else if (since < ST - 2) wait_vmem<(ST - 2) * LPW + NS < 63 ? (ST - 2) * LPW + NS : 63>();
      else wait_vmem<(ST - 2) * LPW>();
      block_barrier();
      const bool now_open = STEADY || open;
      if (now_open) p_rows();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < NMF; ++m) {
#pragma unroll
        for (int f = m * NF / NMF; f < (m + 1) * NF / NMF; ++f) f0[f] = fo.read(base + nxt, 0, f);
        acc[m / TN][m % TN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            f1[TM + m % TN], f1[m / TN], acc[m / TN][m % TN], 0, 0, 0);
        if (now_open) {
#pragma unroll
          for (int j = m * P1 / NMF; j < (m + 1) * P1 / NMF; ++j) p_copy(j, cur);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_lds();
      prv = cur;
      cur = nxt;
      ++since;
    };
    // k-tiles left, and the steady ones among the next
    for (int left = (n + GK - 1) / GK; left > 0;) {
      int steady = open ? min(left, (p_n - p_k - 1) / GK) : 0;
      left -= steady;
      for (; steady > 0; --steady) tile(std::true_type{});
      if (left > 0) {
        tile(std::false_type{});
        --left;
      }
    }
    // the results: 32 rows at a time lie in one matrix (I is a multiple of 32).  The
    // fp32 stores read the accumulators from inline asm: past the last product's 11
    // wait states first
    if constexpr (F32) asm volatile("s_nop 15" ::: "memory");
    const int e = c_it / (MT * NT), mt = c_it / NT % MT, nt = c_it % NT;
    const int n0 = nt * TL::BN;
    const unsigned ldo = (unsigned)N * sizeof(WT);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = mt * TL::BM + wm * WR + i * 32;
      char* p;
      int rows;  // of the matrix, from r on
      if constexpr (KIND == kDWGU) {
        const bool up = r >= I;
        p = static_cast<char*>(up ? o.d_up : o.d_gate) + (size_t)(up ? r - I : r) * ldo +
            (size_t)e * o.gu_stride * sizeof(WT);
        rows = (up ? 2 * I : I) - r;
      } else {
        p = static_cast<char*>(o.d_down) + (size_t)r * ldo +
            (size_t)e * o.dn_stride * sizeof(WT);
        rows = H - r;
      }
      const unsigned first = (unsigned)n0 * sizeof(WT);
      const i32x4 buf = buffer_of(p + first, rows > 0 ? (unsigned)rows * ldo - first : 0u);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int c = wn * WC + j * 32;  // from n0
        if constexpr (F32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int cc = c + 8 * q + 4 * fq;
            const unsigned at = n0 + cc < N ? fr * ldo + cc * 4u : kNowhere;
            const i32x4 v = {__float_as_int(acc[i][j][4 * q]), __float_as_int(acc[i][j][4 * q + 1]),
                             __float_as_int(acc[i][j][4 * q + 2]),
                             __float_as_int(acc[i][j][4 * q + 3])};
            buffer_store16<PAST>(buf, at, v);
          }
        } else {
          // 32 rows of SJ x 32 columns through the wave's own LDS, 16-B chunk q of row r
          // at q ^ f(r), so that 4 SJ lanes store 64 SJ B of a row
          constexpr int SJ = TL::SJ, CPR = 4 * SJ, RPS = 64 / CPR;
          auto place = [](int r, int q) {
            return r * (CPR * 16) + (q ^ (r / (4 / SJ) % CPR)) * 16;
          };
          unsigned char* stg = smem + TL::RING + wave * TL::WAVE_STAGING;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bf16x4 v = {(bf16)acc[i][j][4 * q], (bf16)acc[i][j][4 * q + 1],
                              (bf16)acc[i][j][4 * q + 2], (bf16)acc[i][j][4 * q + 3]};
            *reinterpret_cast<bf16x4*>(stg + place(fr, j % SJ * 4 + q) + fq * 8) = v;
          }
          asm volatile("" ::: "memory");  // the wave's LDS accesses run in order
          if (j % SJ == SJ - 1) {
#pragma unroll
            for (int h = 0; h < 32 / RPS; ++h) {
              const int rr = RPS * h + lane / CPR, ch = lane % CPR;
              const i32x4 v = *reinterpret_cast<const i32x4*>(stg + place(rr, ch));
              const int cc = c - 32 * (SJ - 1) + ch * 8;
              buffer_store16<PAST>(buf, n0 + cc < N ? rr * ldo + cc * 2u : kNowhere, v);
            }
            asm volatile("" ::: "memory");
          }
        }
      }
    }
    since = 0;
  }
}

template <int KIND, typename WT, typename TL, bool PAST>
__global__ __launch_bounds__(64 * TL::NW, TL::WAVES_EU) void grad_weights_kernel(Operands o, int MT,
                                                                                 int NT) {
  extern __shared__ __align__(16) unsigned char smem[];
  weights_block<KIND, WT, TL, PAST>(o, MT, NT, blockIdx.x, gridDim.x, smem);
}

// ---------------------------------------------------------------------------
// fp32 (debug path): BM x 64 tiles on the vector ALUs
// ---------------------------------------------------------------------------
// k-steps of 32, the next one's loads under way while a thread multiplies its
// (BM / 16) x 4 results' operands, both kept k-major in LDS.
constexpr int FN = 64, FK = 32;
template <int KIND>
constexpr int f32_rows() { return KIND == kDWGU || KIND == kDWDN ? 64 : 32; }

template <int KIND>
__device__ __forceinline__ void gemm_f32(const Operands& o, int block, int MT, int NT,
                                         float (*As)[68], float (*Bs)[FN + 4]) {
  constexpr bool DW = KIND == kDWGU || KIND == kDWDN;
  constexpr int BM = f32_rows<KIND>(), TM = BM / 16;
  constexpr int NA = BM * FK / 4 / 256, NB = FN * FK / 4 / 256;  // 16-B loads a thread
  const int H = o.H, I = o.I;
  const int Nout = KIND == kDU || KIND == kDWDN ? I : H;
  const int M = KIND == kDWGU ? 2 * I : H;
  int e = 0, row0, row1, m0 = 0;
  const int nt = block % NT, n0 = nt * FN;
  if constexpr (DW) {
    e = block / (MT * NT);
    m0 = block / NT % MT * BM;
    const bool all = o.ident || o.rows == 0;  // no rows: the offsets may not exist
    row0 = all ? 0 : o.offsets[e];
    row1 = all ? o.rows : o.offsets[e + 1];
  } else if (o.ident) {
    row0 = block / NT * BM;
    row1 = min(row0 + BM, o.rows);
  } else if (!find_row_tile(o.offsets, o.E, BM, block / NT, e, row0, row1)) {
    return;  // uniform over the block
  }
  const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
  const float* d_out = static_cast<const float*>(o.d_out);
  const float* x = static_cast<const float*>(o.x);
  const float* kept = static_cast<const float*>(o.kept);
  if (KIND == kDU && nt == 0) write_tables(o, row0, row1, 4u * (unsigned)H);
  auto row_of = [&](const float* p, unsigned off) {  // a token's
    return reinterpret_cast<const float*>(reinterpret_cast<const char*>(p) + off);
  };
  int toks[NA];  // DU: the tokens of this thread's rows
#pragma unroll
  for (int u = 0; u < NA && KIND == kDU; ++u) {
    const int r = row0 + (threadIdx.x + 256 * u) / (FK / 4);
    toks[u] = r < row1 ? token_of(o, r) : -1;
  }
  float* d_gu = static_cast<float*>(o.d_gu);
  float* hw = static_cast<float*>(o.hw);
  const float* wg = static_cast<const float*>(o.w_gate) + (size_t)e * o.gu_stride;
  const float* wu = static_cast<const float*>(o.w_up) + (size_t)e * o.gu_stride;
  const float* wd = static_cast<const float*>(o.w_down) + (size_t)e * o.dn_stride;
  const int Kd = DW ? row1 - row0 : KIND == kDU ? H : 2 * I;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  auto ld4 = [](const float* p) { return *reinterpret_cast<const f32x4*>(p); };

  f32x4 va[NA], vb[NB];
  auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < NA; ++u) {
      const int i = tid + 256 * u;
      va[u] = zero;
      if constexpr (DW) {
        const int k = k0 + i / (BM / 4), c = m0 + i % (BM / 4) * 4, r = row0 + k;
        if (k < Kd && c < M) {
          const unsigned off = o.row_off[r];
          if (off != kNowhere)
            va[u] = ld4(KIND == kDWGU ? d_gu + (size_t)r * 2 * I + c : row_of(d_out, off) + c);
        }
      } else {
        const int r = row0 + i / (FK / 4), k = k0 + i % (FK / 4) * 4;  // Kd is a multiple of 32
        if (r < row1) {
          if constexpr (KIND == kDU) {
            if (toks[u] >= 0) va[u] = ld4(d_out + (size_t)toks[u] * H + k);
          } else {
            va[u] = ld4(d_gu + (size_t)r * 2 * I + k);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const int i = tid + 256 * u, k = k0 + i / (FN / 4), c = n0 + i % (FN / 4) * 4;
      vb[u] = zero;
      if (k >= Kd || c >= Nout) continue;
      if constexpr (KIND == kDU) {
        vb[u] = ld4(wd + (size_t)k * I + c);
      } else if constexpr (KIND == kDX) {
        vb[u] = ld4(k < I ? wg + (size_t)k * H + c : wu + (size_t)(k - I) * H + c);
      } else {
        const int r = row0 + k;
        const unsigned off = o.row_off[r];
        if (off != kNowhere)
          vb[u] = ld4(KIND == kDWGU ? row_of(x, off) + c : hw + (size_t)r * I + c);
      }
    }
  };
  float acc[TM][4] = {};
  if (Kd > 0) load(0);
  for (int k0 = 0; k0 < Kd; k0 += FK) {
#pragma unroll
    for (int u = 0; u < NA; ++u) {
      const int i = tid + 256 * u;
      if constexpr (DW) {
        *reinterpret_cast<f32x4*>(&As[i / (BM / 4)][i % (BM / 4) * 4]) = va[u];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) As[i % (FK / 4) * 4 + j][i / (FK / 4)] = va[u][j];
      }
    }
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const int i = tid + 256 * u;
      *reinterpret_cast<f32x4*>(&Bs[i / (FN / 4)][i % (FN / 4) * 4]) = vb[u];
    }
    __syncthreads();
    if (k0 + FK < Kd) load(k0 + FK);
#pragma unroll
    for (int k = 0; k < FK; ++k) {
      const f32x4 b = ld4(&Bs[k][4 * tc]);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][TM * tr + i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int rl = TM * tr + i, row = row0 + rl, col = n0 + 4 * tc;
    const bool in = col < Nout;  // four columns are inside or outside together
    const f32x4 v = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
    if constexpr (KIND == kDU) {
      float dot = 0.0f;
      if (row < row1 && in) {
        const bool live = token_of(o, row) >= 0;
        const float w = o.ident ? 1.0f : o.topk_w[o.sorted_slots[row]];
        const f32x4 g = ld4(kept + (size_t)row * 2 * I + col);
        const f32x4 u = ld4(kept + (size_t)row * 2 * I + I + col);
        f32x4 og = zero, ou = zero, oh = zero;
        if (live) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float h, dg, du;
            act_grad<false>(g[j], u[j], v[j], h, dg, du);
            dot += v[j] * h;
            og[j] = w * dg;
            ou[j] = w * du;
            oh[j] = w * h;
          }
        }
        *reinterpret_cast<f32x4*>(d_gu + (size_t)row * 2 * I + col) = og;
        *reinterpret_cast<f32x4*>(d_gu + (size_t)row * 2 * I + I + col) = ou;
        *reinterpret_cast<f32x4*>(hw + (size_t)row * I + col) = oh;
      }
      if (o.part) {
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) dot += __shfl_xor(dot, s, kWave);
        if (tc == 0 && row < row1) o.part[(size_t)nt * o.rows + row] = dot;
      }
    } else if constexpr (KIND == kDX) {
      if (row < row1 && in)
        *reinterpret_cast<f32x4*>(static_cast<float*>(o.d_xs) + (size_t)row * H + col) = v;
    } else {
      const int m = m0 + rl;
      if (m < M && in) {
        float* d;
        if constexpr (KIND == kDWGU)
          d = (m < I ? static_cast<float*>(o.d_gate) + (size_t)m * H
                     : static_cast<float*>(o.d_up) + (size_t)(m - I) * H) +
              (size_t)e * o.gu_stride;
        else
          d = static_cast<float*>(o.d_down) + (size_t)e * o.dn_stride + (size_t)m * I;
        *reinterpret_cast<f32x4*>(d + col) = v;
      }
    }
  }
}

__global__ __launch_bounds__(256) void grad_du_f32_kernel(Operands o, int NT) {
  __shared__ __align__(16) float As[FK][68], Bs[FK][FN + 4];
  gemm_f32<kDU>(o, blockIdx.x, 0, NT, As, Bs);
}

// The other three, which need DU alone, in one launch (100 tokens, 12 experts of 320 x
// 224: 21 us, one after another 36).
struct F32Tiles { int dx, dwgu, end; };  // first block behind DX's, behind DWGU's, of all
__global__ __launch_bounds__(256) void grad_rest_f32_kernel(Operands o, F32Tiles n) {
  __shared__ __align__(16) float As[FK][68], Bs[FK][FN + 4];
  const int NH = (o.H + FN - 1) / FN, NI = (o.I + FN - 1) / FN;
  const int b = blockIdx.x;
  if (b < n.dx) gemm_f32<kDX>(o, b, 0, NH, As, Bs);
  else if (b < n.dwgu) gemm_f32<kDWGU>(o, b - n.dx, (2 * o.I + 63) / 64, NH, As, Bs);
  else gemm_f32<kDWDN>(o, b - n.dwgu, NH, NI, As, Bs);
}

// DU and DX: 128 x 256, two blocks of 8 waves a CU; DW: 256 x 256, one block of 8
// waves, four stages (26B-A4B at 64 / 4096 tokens, DWGU + DWDN 298 / 745 us; 128 x 256 in
// two blocks of 4 waves a CU 473 / 939, waves of 64 x 128 303 / 744).
typedef Tile<128, 256, 2, 4, 3, 2> RowsTile;
typedef Tile<256, 256, 2, 4, 4, 1> WeightsTile;
// DU and DX of small problems: 64 x 64, the contraction split over 8 single waves.
typedef Tile<64, 64, 1, 1, 2, 1> FewTile;
constexpr int kFewSplit = 8;
// DW of small problems: 128 x 128, two blocks of 4 waves a CU.
typedef Tile<128, 128, 2, 2, 3, 2> SmallWeightsTile;
constexpr int kCUs = 256;


// The dense MLP's DX, DWGU and DWDN in one launch: DX's blocks in the small form, then a
// large tile a block.  2816 x 2112 at 301 tokens 41 us; one after another 26 + 17 + 11.
struct RestBlocks { int dx, gu, end; };  // behind DX's, behind DWGU's, all; multiples of 8
template <typename WT>
__global__ __launch_bounds__(512, 2) void grad_rest_kernel(Operands o, RestBlocks n) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int BM = WeightsTile::BM, BN = WeightsTile::BN;
  const int b = blockIdx.x;
  if (b < n.dx)
    rows_block<kDX, bf16, FewTile, kFewSplit, false>(o, (o.H + FewTile::BN - 1) / FewTile::BN, b,
                                                     smem);
  else if (b < n.gu)
    weights_block<kDWGU, WT, WeightsTile, false>(o, (2 * o.I + BM - 1) / BM, (o.H + BN - 1) / BN,
                                                 b - n.dx, n.gu - n.dx, smem);
  else
    weights_block<kDWDN, WT, WeightsTile, false>(o, (o.H + BM - 1) / BM, (o.I + BN - 1) / BN,
                                                 b - n.gu, n.end - n.gu, smem);
}

template <int KIND, typename WT, typename TL, int KS, bool ONCE>
hipError_t launch_rows(const FfnGradArgs& a, const Operands& o, hipStream_t s) {
  const int NT = ((KIND == kDU ? a.I : a.H) + TL::BN - 1) / TL::BN;
  const int blocks = tile_count_bound(a.ident, a.rows, a.T, a.E, TL::BM) * NT;
  auto kf = grad_rows_kernel<KIND, WT, TL, KS, ONCE>;
  constexpr int lds = TL::template rows_lds<KS>();
  static_assert(TL::BLOCKS * lds <= 160 * 1024, "LDS");
  static const hipError_t attr = hipFuncSetAttribute(
      reinterpret_cast<const void*>(kf), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kf, dim3(blocks), dim3(64 * TL::NW * KS), lds, s, o, NT);
  return hipGetLastError();
}

// Whether DU (N = I) or DX (N = H) takes the small form: while its blocks, one a CU,
// are one and a half a CU at most.  The dense MLP (2816 x 2112) at 16 / 301 / 700 /
// 1200 tokens, DU: 14 / 20 / 38 / 58 us, in the large form 28 / 46 / 48 / 48; DX 16 /
// 26 / 52 / 98 and 36 / 49 / 51 / 53.  (128 x 128 tiles split over four groups of
// four waves: DU 24 / 36 / 38 / 40.)
bool small_rows(const FfnGradArgs& a, int N) {
  return tile_count_bound(a.ident, a.rows, a.T, a.E, FewTile::BM) *
             ((N + FewTile::BN - 1) / FewTile::BN) <= kCUs * 3 / 2;
}

template <int KIND, typename WT, typename TL, bool PAST>
hipError_t launch_weights(const FfnGradArgs& a, const Operands& o, hipStream_t s) {
  const int N = KIND == kDWDN ? a.I : a.H, M = KIND == kDWGU ? 2 * a.I : a.H;
  const int NT = (N + TL::BN - 1) / TL::BN, MT = (M + TL::BM - 1) / TL::BM;
  const int tiles = o.E * MT * NT;
  auto kf = grad_weights_kernel<KIND, WT, TL, PAST>;
  constexpr int lds = TL::RING + TL::NW * TL::WAVE_STAGING;
  static_assert(TL::BLOCKS * lds <= 160 * 1024, "LDS");
  static const hipError_t attr = hipFuncSetAttribute(
      reinterpret_cast<const void*>(kf), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return attr;
  const int most = kCUs * TL::BLOCKS, blocks = tiles < most ? (tiles + 7) / 8 * 8 : most;
  hipLaunchKernelGGL(kf, dim3(blocks), dim3(64 * TL::NW), lds, s, o, MT, NT);
  return hipGetLastError();
}

template <int KIND, typename WT>
hipError_t launch_gemm(const FfnGradArgs& a, const Operands& o, hipStream_t s) {
  constexpr bool DW = KIND == kDWGU || KIND == kDWDN;
  const int N = KIND == kDU || KIND == kDWDN ? a.I : a.H;
  const int M = KIND == kDWGU ? 2 * a.I : a.H;
  if constexpr (DW) {
    const int tiles = o.E * ((M + WeightsTile::BM - 1) / WeightsTile::BM) *
                      ((N + WeightsTile::BN - 1) / WeightsTile::BN);
    // Up to half as many large tiles as CUs: the dense MLP's DWDN (99 tiles) at 301 / 4096
    // tokens 14.0 / 93 -> 10.7 / 63 us; its DWGU (187) 16.6 / 106, with small ones 16.0 / 121.
    if (tiles <= kCUs / 2) return launch_weights<KIND, WT, SmallWeightsTile, false>(a, o, s);
    // All three gradients in bf16, a quarter of the last cache or more: past it.  512 tokens
    // x 2, 2816 x 704, the call alone with 8 / 16 / 32 experts (95 / 190 / 381 MB) 91 / 106 /
    // 192 us, through the caches 93 / 137 / 201; with the norm and the clipping of them
    // behind it, which find up to 190 MB in the caches, 145 / 228 / 387 and 143 / 223 / 409.
    // The dense MLP (36 MB) at 4096 tokens 346 and 351, with both 373 and 371.
    // fp32 ones go through the caches, which join a store's 32-byte pieces of a row to lines;
    // past them each is written by itself: 512 tokens x 8 with 16 / 32 experts (DWGU + DWDN)
    // 141 and 424 / 225 and 833 us, 26B-A4B at 64 / 4096 tokens 582 and 3471 / 1062 and 3285.
    if constexpr (std::is_same<WT, bf16>::value) {
      const long long bytes = (long long)o.E * 3 * o.I * o.H * sizeof(WT);
      if (bytes >= 64 << 20) return launch_weights<KIND, WT, WeightsTile, true>(a, o, s);
    }
    return launch_weights<KIND, WT, WeightsTile, false>(a, o, s);
  } else {
    if (small_rows(a, N)) return launch_rows<KIND, WT, FewTile, kFewSplit, false>(a, o, s);
    // Up to 32 rows an expert on average most have one row tile, which reads the weights
    // alone.  26B-A4B at 64 / 256 / 512 / 1024 / 4096 tokens, DU 90 / 107 / 136 / 157 / 335
    // us, with copies that stay 95 / 116 / 136 / 154 / 289; DX 128 / 167 / 190 / 231 / 496
    // and 149 / 182 / 197 / 230 / 380.
    if (!a.ident && (long long)a.rows <= 32LL * a.E)
      return launch_rows<KIND, WT, RowsTile, 1, true>(a, o, s);
    return launch_rows<KIND, WT, RowsTile, 1, false>(a, o, s);
  }
}

template <typename XT, typename ST>
void launch_combine_grad(const FfnGradArgs& a, int parts, hipStream_t s) {
  hipLaunchKernelGGL((combine_grad_kernel<XT, ST>), dim3(a.T), dim3(256), 0, s, a.T, a.H, a.K, a.E,
                     parts, (long long)a.rows, a.offsets, a.sorted_slots, a.ws_slot_row,
                     static_cast<const ST*>(a.ws_d_xs), a.ws_part, static_cast<XT*>(a.d_x),
                     a.d_topk_w);
}

hipError_t launch_combine(const FfnGradArgs& a, hipStream_t s) {
  if (a.ident || a.rows == 0 || !(a.d_x || a.d_topk_w)) return hipSuccess;
  const int pn = !a.bf16 ? FN : small_rows(a, a.I) ? FewTile::BN : RowsTile::BN;
  const int parts = (a.I + pn - 1) / pn;
  if (!a.bf16) launch_combine_grad<float, float>(a, parts, s);
  else if (a.xs_bf16) launch_combine_grad<bf16, bf16>(a, parts, s);
  else launch_combine_grad<bf16, float>(a, parts, s);
  return hipGetLastError();
}

hipError_t launch_f32(const FfnGradArgs& a, const Operands& o, hipStream_t s) {
  const int RT = a.rows > 0 ? tile_count_bound(a.ident, a.rows, a.T, a.E, f32_rows<kDX>()) : 0;
  const int NH = (a.H + FN - 1) / FN, NI = (a.I + FN - 1) / FN;
  if (RT > 0) {
    hipLaunchKernelGGL(grad_du_f32_kernel, dim3(RT * NI), dim3(256), 0, s, o, NI);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  F32Tiles n;
  n.dx = a.d_x ? RT * NH : 0;
  n.dwgu = n.dx + (a.d_gate ? o.E * ((2 * a.I + 63) / 64) * NH : 0);
  n.end = n.dwgu + (a.d_down ? o.E * NH * NI : 0);
  if (n.end > 0) {
    hipLaunchKernelGGL(grad_rest_f32_kernel, dim3(n.end), dim3(256), 0, s, o, n);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_combine(a, s);
}

template <typename WT>
hipError_t launch_rest(const FfnGradArgs& a, const Operands& o, hipStream_t s) {
  typedef WeightsTile W;
  auto eights = [](int n) { return (n + 7) / 8 * 8; };
  auto over = [](int n, int d) { return (n + d - 1) / d; };
  RestBlocks n;
  n.dx = eights(over(a.rows, FewTile::BM) * over(a.H, FewTile::BN));
  n.gu = n.dx + (a.d_gate ? eights(over(2 * a.I, W::BM) * over(a.H, W::BN)) : 0);
  n.end = n.gu + (a.d_down ? eights(over(a.H, W::BM) * over(a.I, W::BN)) : 0);
  auto kf = grad_rest_kernel<WT>;
  constexpr int wlds = W::RING + W::NW * W::WAVE_STAGING, rlds = FewTile::rows_lds<kFewSplit>();
  constexpr int lds = wlds > rlds ? wlds : rlds;
  static_assert(lds <= 160 * 1024 && W::NW == 8 && kFewSplit * FewTile::NW == 8, "one block shape");
  static const hipError_t attr = hipFuncSetAttribute(
      reinterpret_cast<const void*>(kf), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kf, dim3(n.end), dim3(512), lds, s, o, n);
  return hipGetLastError();
}

hipError_t launch_bf16(const FfnGradArgs& a, const Operands& o, hipStream_t s) {
  hipError_t e;
  if (a.rows > 0) {
    if ((e = launch_gemm<kDU, bf16>(a, o, s)) != hipSuccess) return e;
    // (small enough for the small form: few blocks, which would leave CUs without work)
    if (a.ident && a.d_x && (a.d_gate || a.d_down) && small_rows(a, a.H))
      return a.wgrad_bf16 ? launch_rest<bf16>(a, o, s) : launch_rest<float>(a, o, s);
    if (a.d_x) {
      e = a.ident || a.xs_bf16 ? launch_gemm<kDX, bf16>(a, o, s) : launch_gemm<kDX, float>(a, o, s);
      if (e != hipSuccess) return e;
    }
    // behind DX, whose results are in the caches still: 51 us at 4096 tokens, at the
    // end 80
    if ((e = launch_combine(a, s)) != hipSuccess) return e;
  }
  const bool b = a.wgrad_bf16;
  if (a.d_gate) {
    e = b ? launch_gemm<kDWGU, bf16>(a, o, s) : launch_gemm<kDWGU, float>(a, o, s);
    if (e != hipSuccess) return e;
  }
  if (!a.d_down) return hipSuccess;
  return b ? launch_gemm<kDWDN, bf16>(a, o, s) : launch_gemm<kDWDN, float>(a, o, s);
}

}  // namespace

// Partial sums of d_topk_w: DU's column tiles, those of its widest grid.
int ffn_grad_parts(int I, bool bf16) {
  const int n = bf16 ? FewTile::BN : FN;
  return (I + n - 1) / n;
}

hipError_t launch_ffn_grad(const FfnGradArgs& a, hipStream_t s) {
  Operands o{};
  o.T = a.T; o.H = a.H; o.I = a.I; o.E = a.ident ? 1 : a.E; o.K = a.K;
  o.rows = a.rows; o.ident = a.ident;
  o.offsets = a.offsets; o.sorted_slots = a.sorted_slots; o.mask = a.mask;
  o.row_off = a.ws_row_off; o.slot_row = a.ws_slot_row;
  o.topk_w = a.topk_w; o.x = a.x; o.d_out = a.d_out; o.kept = a.kept;
  o.w_gate = a.w_gate; o.w_up = a.w_up; o.w_down = a.w_down;
  o.gu_stride = a.gu_stride; o.dn_stride = a.dn_stride;
  o.d_gu = a.ws_d_gu; o.hw = a.ws_hw; o.part = a.d_topk_w ? a.ws_part : nullptr;
  o.d_xs = a.ident ? a.d_x : a.ws_d_xs;
  o.d_gate = a.d_gate; o.d_up = a.d_up; o.d_down = a.d_down;
  return a.bf16 ? launch_bf16(a, o, s) : launch_f32(a, o, s);
}

}  // namespace moe
