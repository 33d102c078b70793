// C ABI of libmoe (declared in include/moe.h): host-side argument checks,
// workspace layout, and the kernel sequence of each call on the caller's
// stream.  No call synchronises or allocates.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <string>

#include "../../include/moe.h"
#include "launch.h"

namespace {

thread_local std::string g_err;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return code;
}

int hip_fail(hipError_t e, const char* where) {
  return fail(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

constexpr int32_t kMaxGradTensors = 1 << 16;
constexpr int64_t kMaxGradElements = (int64_t)1 << 40;

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

size_t dtype_size(int32_t dt) { return dt == MOE_BF16 ? 2 : 4; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// any_k: calls that only see token-slots (experts, combine) take any top_k up
// to num_experts, e.g. every expert per token; routing needs top_k <= 32.
int check_dims(const moe_dims* d, bool any_k = false) {
  if (!d) return fail(MOE_ERR_ARG, "dims is NULL");
  if (d->hidden < 64 || d->hidden > 8192 || d->hidden % 64)
    return fail(MOE_ERR_UNSUPPORTED, "hidden=%d: need a multiple of 64 in [64, 8192]", d->hidden);
  if (d->num_experts < 1 || d->num_experts > 256)
    return fail(MOE_ERR_UNSUPPORTED, "num_experts=%d: need 1..256", d->num_experts);
  if (d->top_k < 1 || d->top_k > d->num_experts || (!any_k && d->top_k > 32))
    return fail(MOE_ERR_UNSUPPORTED, "top_k=%d: need 1..min(num_experts, %d)", d->top_k,
                any_k ? d->num_experts : 32);
  if (d->expert_inter < 32 || d->expert_inter > 8192 || d->expert_inter % 32)
    return fail(MOE_ERR_UNSUPPORTED, "expert_inter=%d: need a multiple of 32 in [32, 8192]",
                d->expert_inter);
  if (d->dense_inter < 0 || d->dense_inter > 16384 || d->dense_inter % 32)
    return fail(MOE_ERR_UNSUPPORTED, "dense_inter=%d: need 0 or a multiple of 32 up to 16384",
                d->dense_inter);
  if (!(d->eps > 0.0f)) return fail(MOE_ERR_ARG, "eps must be > 0");
  if (d->act_dtype != MOE_F32 && d->act_dtype != MOE_BF16)
    return fail(MOE_ERR_ARG, "act_dtype=%d unknown", d->act_dtype);
  if (d->slot_dtype != MOE_F32 && d->slot_dtype != MOE_BF16)
    return fail(MOE_ERR_ARG, "slot_dtype=%d unknown", d->slot_dtype);
  if (d->act_dtype == MOE_F32 && d->slot_dtype != MOE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "act_dtype F32 requires slot_dtype F32");
  return MOE_OK;
}

int check_tokens(const moe_dims* d, int32_t T) {
  if (T < 0 || T > 65536) return fail(MOE_ERR_ARG, "T=%d: need 0..65536", T);
  if ((long long)T * d->top_k > (1 << 20))
    return fail(MOE_ERR_UNSUPPORTED, "T*top_k=%lld exceeds 2^20", (long long)T * d->top_k);
  return MOE_OK;
}

#define REQUIRE_PTR(p)                                                                   \
  do {                                                                                   \
    if (!(p)) return fail(MOE_ERR_ARG, "%s is NULL", #p);                                \
    if (!aligned16(p)) return fail(MOE_ERR_ARG, "%s is not 16-byte aligned", #p);        \
  } while (0)
#define OPTIONAL_PTR(p)                                                                  \
  do {                                                                                   \
    if ((p) && !aligned16(p)) return fail(MOE_ERR_ARG, "%s is not 16-byte aligned", #p); \
  } while (0)

// The next region of a workspace: its offset, with `o` moved past it.
size_t region(size_t& o, size_t bytes) {
  const size_t at = o;
  o += align256(bytes);
  return at;
}

// Workspace regions (byte offsets), all 256-byte aligned, monotone in T so
// that a workspace sized for max_tokens serves every T <= max_tokens.
struct Layout {
  size_t r0, r, logits;             // router
  size_t blk_counts, local_rank;    // dispatch
  size_t h;                         // expert gate_up output
  size_t idx, w, counts, offsets, sorted, y;  // experts-only path / layer
  size_t xd, xm, hd, dn;            // layer only
  size_t counter;                   // small-batch top-K completion counter
  size_t base_end;                  // end of the regions above (all but the MXFP8 ones)
  size_t xq, xs, hq, hs;            // MXFP8 activations of the 8-bit / 4-bit experts
  size_t total;
};

Layout layout(const moe_dims* d, long long T) {
  Layout L{};
  const long long S = T * d->top_k;
  const long long nblk = (S + 1023) / 1024;
  const size_t act = dtype_size(d->act_dtype), slot = dtype_size(d->slot_dtype);
  size_t o = 0;
  auto take = [&](size_t bytes) { return region(o, bytes); };
  L.r0 = take(4 * T);
  L.r = take(4 * T);
  L.logits = take(4 * T * d->num_experts);
  L.blk_counts = take(4 * nblk * d->num_experts);
  L.local_rank = take(4 * S);
  L.h = take(act * S * d->expert_inter);
  L.idx = take(4 * S);
  L.w = take(4 * S);
  L.counts = take(4 * (size_t)d->num_experts);
  L.offsets = take(4 * (size_t)(d->num_experts + 1));
  L.sorted = take(4 * S);
  L.y = take(slot * S * d->hidden);
  L.xd = take(act * T * d->hidden);
  L.xm = take(act * T * d->hidden);
  L.hd = take(act * T * d->dense_inter);
  L.dn = take(slot * T * d->hidden);
  L.counter = take(4);
  L.base_end = o;
  L.xq = take((size_t)T * d->hidden);
  L.xs = take((size_t)T * (d->hidden / 32));
  L.hq = take((size_t)S * d->expert_inter);
  L.hs = take((size_t)S * (d->expert_inter / 32));
  L.total = o;
  return L;
}

// The training calls and the block-scaled experts have workspaces of sizes of
// their own: part of the layout above, their scratch would be asked of every
// call (at 26B-A4B and one token 3.1 MB instead of 0.14).  Their regions start
// at the workspace's first byte and hold nothing between calls, so a balance
// loss of 65536 tokens asks for 0.3 MB, not for a layer's 9 GB beside it.
struct BalanceLayout { size_t p, n, z, live, total; };
BalanceLayout balance_layout(const moe_dims* d, long long T) {
  BalanceLayout L{};
  const size_t E = (size_t)d->num_experts, nb = (size_t)moe::balance_blocks((int)T);
  size_t o = 0;
  L.p = region(o, 4 * nb * E);
  L.n = region(o, 4 * nb * E);
  L.z = region(o, 4 * nb);
  L.live = region(o, 4 * nb);
  L.total = o;
  return L;
}

struct RouterGradLayout { size_t dl, beta, g, b, pes, total; };
RouterGradLayout router_grad_layout(const moe_dims* d, long long T) {
  RouterGradLayout L{};
  const size_t E = (size_t)d->num_experts, H = (size_t)d->hidden;
  const size_t splits = (size_t)moe::router_grad_max_splits((int)T, d->hidden, d->num_experts);
  size_t o = 0;
  L.dl = region(o, moe::router_grad_dl_bytes((int)T, d->hidden, d->num_experts));
  L.beta = region(o, 4 * (((size_t)T + 31) / 32 * 32));
  L.g = region(o, 4 * splits * E * H);
  L.b = region(o, 4 * splits * H);
  L.pes = region(o, 4 * (size_t)moe::router_grad_row_blocks((int)T) * E);
  L.total = o;
  return L;
}

struct B128Layout { size_t xq, xs, h, hq, hs, total; };
B128Layout b128_layout(const moe_dims* d, long long T) {
  B128Layout L{};
  const size_t H = (size_t)d->hidden, I = (size_t)d->expert_inter, S = (size_t)T * d->top_k;
  const size_t ts = (size_t)(T < moe::kB128StreamTokens ? T : moe::kB128StreamTokens);
  size_t o = 0;
  L.xq = region(o, (size_t)T * ((H + 127) / 128 * 128));
  L.xs = region(o, 4 * (size_t)T * ((H + 127) / 128));
  L.h = region(o, 4 * ts * d->top_k * I);  // fp32, the weight-streaming form only
  L.hq = region(o, S * ((I + 127) / 128 * 128));
  L.hs = region(o, 4 * S * ((I + 127) / 128));
  L.total = o + 256;  // never 0, which says that the sizes are not supported
  return L;
}

// Backward pass of the gated block over `rows` rows of width I.
struct FfnGradLayout { size_t row_off, slot_row, d_gu, hw, d_xs, part, total; };
FfnGradLayout ffn_grad_layout(const moe_dims* d, long long rows, long long I, bool experts) {
  FfnGradLayout L{};
  const bool bf = d->act_dtype == MOE_BF16;
  const size_t act = dtype_size(d->act_dtype), S = (size_t)rows;
  size_t o = 0;
  L.row_off = region(o, 4 * (S + 32));
  L.slot_row = region(o, experts ? 4 * S : 0);
  L.d_gu = region(o, act * S * 2 * I);
  L.hw = region(o, act * S * I);
  L.d_xs = region(o, experts ? dtype_size(d->slot_dtype) * S * d->hidden : 0);
  L.part = region(o, experts ? 4 * S * moe::ffn_grad_parts((int)I, bf) : 0);
  L.total = o + 256;  // never 0, which says that the sizes are not supported
  return L;
}

struct NormsGradLayout { size_t scalar, part, total; };
NormsGradLayout norms_grad_layout(const moe_dims* d, long long T) {
  NormsGradLayout L{};
  const size_t nb = (size_t)moe::norms_grad_blocks((int)T, d->hidden, d->slot_dtype == MOE_BF16);
  size_t o = 0;
  L.scalar = region(o, 8 * nb);
  L.part = region(o, 4 * nb * 3 * d->hidden);
  L.total = o + 256;
  return L;
}

// The block's dense branch runs on a library-owned side stream (one per
// device, default priority, created on first use and kept), forked from and
// joined back into the caller's stream with two events.  A mutex keeps one
// call's record / wait sequence from interleaving with another thread's.
struct SideStream {
  hipStream_t stream = nullptr;
  hipEvent_t fork = nullptr, join = nullptr;
};
std::mutex g_side_mu;
SideStream g_side[64];

hipError_t side_stream(SideStream*& out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
  SideStream& ss = g_side[dev];
  if (ss.stream == nullptr) {
    if ((e = hipStreamCreateWithFlags(&ss.stream, hipStreamNonBlocking)) != hipSuccess) return e;
    if ((e = hipEventCreateWithFlags(&ss.fork, hipEventDisableTiming)) != hipSuccess) return e;
    if ((e = hipEventCreateWithFlags(&ss.join, hipEventDisableTiming)) != hipSuccess) return e;
  }
  out = &ss;
  return hipSuccess;
}

template <typename P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

int check_ws(size_t need, const char* what, const void* ws, size_t ws_bytes) {
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(MOE_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed for %s", ws_bytes, need,
                what);
  return MOE_OK;
}
int check_ws(size_t need, int32_t T, const void* ws, size_t ws_bytes) {
  char what[24];
  snprintf(what, sizeof(what), "T=%d", T);
  return check_ws(need, what, ws, ws_bytes);
}
int check_ws(const moe_dims* d, int32_t T, const void* ws, size_t ws_bytes) {
  return check_ws(layout(d, T).total, T, ws, ws_bytes);
}

// ---- scratch of the entry point that allocates nothing --------------------
// moe_forward_noalloc takes its workspace from this file-scope device array
// instead of a caller's buffer.  Each GPU the library runs on holds its own
// copy until the process ends.  In host code the array's name is only a
// host-side stand-in: the device address of a GPU's copy comes from
// hipGetSymbolAddress, taken once per device (with that device current) and
// kept; only that address is ever handed to kernels.  Every call on a GPU
// shares the array and finds the last call's contents; the path clears what
// it needs cleared itself (the router's completion counter is zeroed by its
// logits kernel), and calls that overlap on one GPU race.
constexpr size_t kNoAllocScratchBytes = size_t(64) << 20;
__device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_ptr[64];

hipError_t noalloc_scratch(void*& out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* p = nullptr;
    if ((e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch))) != hipSuccess) return e;
    if (p == nullptr) return hipErrorInvalidSymbol;
    g_scratch_ptr[dev] = p;
  }
  out = g_scratch_ptr[dev];
  return hipSuccess;
}

int run_forward(const moe_dims* dims, int32_t T, const void* x, const float* router_w,
                const float* router_scale, const float* per_expert_scale,
                const void* w_gate_up, const void* w_down, void* out, int32_t* topk_idx,
                float* topk_w, void* ws, hipStream_t s);

// ---- launch sequences (arguments already checked) -------------------------

// Router, and when counts is not null the dispatch as well (fused into the
// router's top-K kernel for small batches).
int run_router(const moe_dims* d, int32_t T, const void* x, const float* router_w,
               const float* router_scale, const float* pes, const float* pre_gain,
               int32_t* idx, float* w, int32_t* counts, int32_t* offsets, int32_t* sorted,
               void* ws, hipStream_t s, float* logits = nullptr) {
  const Layout L = layout(d, T);
  moe::RouterArgs a{};
  a.T = T; a.H = d->hidden; a.E = d->num_experts; a.K = d->top_k; a.eps = d->eps;
  a.x_bf16 = d->act_dtype == MOE_BF16;
  a.x = x; a.pre_gain = pre_gain; a.router_w = router_w; a.router_scale = router_scale;
  a.per_expert_scale = pes; a.topk_idx = idx; a.topk_w = w;
  a.ws_r0 = at<float>(ws, L.r0); a.ws_r = at<float>(ws, L.r);
  a.ws_logits = logits ? logits : at<float>(ws, L.logits);
  a.ws_counter = at<unsigned>(ws, L.counter);
  a.counts = counts; a.offsets = offsets; a.sorted_slots = sorted;
  a.ws_blk_counts = at<int32_t>(ws, L.blk_counts);
  a.ws_local_rank = at<int32_t>(ws, L.local_rank);
  hipError_t e = moe::launch_router(a, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e, counts ? "moe_route" : "moe_router");
}

int run_dispatch(const moe_dims* d, int32_t T, const int32_t* idx, int32_t* counts,
                 int32_t* offsets, int32_t* sorted, void* ws, hipStream_t s) {
  const Layout L = layout(d, T);
  moe::DispatchArgs a{};
  a.T = T; a.E = d->num_experts; a.K = d->top_k;
  a.topk_idx = idx; a.counts = counts; a.offsets = offsets; a.sorted_slots = sorted;
  a.ws_blk_counts = at<int32_t>(ws, L.blk_counts);
  a.ws_local_rank = at<int32_t>(ws, L.local_rank);
  hipError_t e = moe::launch_dispatch(a, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_dispatch");
}

int run_gate_up(const moe_dims* d, int32_t T, const void* x, const void* w_gate_up,
                const int32_t* offsets, const int32_t* sorted, void* h, hipStream_t s,
                hipEvent_t ev_start = nullptr, hipEvent_t ev_stop = nullptr,
                void* keep = nullptr) {
  const size_t act = dtype_size(d->act_dtype);
  const long long H = d->hidden, I = d->expert_inter;
  moe::GateUpArgs g{};
  g.T = T; g.H = d->hidden; g.N = d->expert_inter; g.E = d->num_experts; g.K = d->top_k;
  g.rows = T * d->top_k; g.ident = false; g.bf16 = d->act_dtype == MOE_BF16;
  g.x = x;
  g.w_gate = w_gate_up;
  g.w_up = static_cast<const char*>(w_gate_up) + act * I * H;
  g.w_stride = 2 * I * H;
  g.offsets = offsets; g.sorted_slots = sorted; g.h = h; g.keep = keep;
  g.ev_start = ev_start; g.ev_stop = ev_stop;
  hipError_t e = moe::launch_gate_up(g, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "expert gate_up");
}

int run_down(const moe_dims* d, int32_t T, const void* h, const void* w_down,
             const float* topk_w, const int32_t* offsets, const int32_t* sorted, void* y,
             hipStream_t s) {
  moe::DownArgs dn{};
  dn.T = T; dn.H = d->hidden; dn.N = d->expert_inter; dn.E = d->num_experts; dn.K = d->top_k;
  dn.rows = T * d->top_k; dn.ident = false; dn.bf16 = d->act_dtype == MOE_BF16;
  dn.y_bf16 = d->slot_dtype == MOE_BF16;
  dn.h = h; dn.w_down = w_down; dn.w_stride = (long long)d->hidden * d->expert_inter;
  dn.offsets = offsets; dn.sorted_slots = sorted; dn.topk_w = topk_w; dn.y = y;
  hipError_t e = moe::launch_down(dn, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "expert down");
}

int run_expert_ffn(const moe_dims* d, int32_t T, const void* x, const void* w_gate_up,
                   const void* w_down, const float* topk_w, const int32_t* offsets,
                   const int32_t* sorted, void* y, void* ws, hipStream_t s,
                   void* keep = nullptr) {
  void* h = at<void>(ws, layout(d, T).h);
  int rc = run_gate_up(d, T, x, w_gate_up, offsets, sorted, h, s, nullptr, nullptr, keep);
  if (rc) return rc;
  return run_down(d, T, h, w_down, topk_w, offsets, sorted, y, s);
}

// Experts on weights stored below bf16 (fmt: int8, E4M3 or MXFP4).  Codes
// of gate_up are [E, 2I, H] and of down [E, H, I] (MXFP4: two per byte);
// scales are fp32 [E, 2I] / [E, H] (int8, E4M3) or E8M0 [E, 2I, H/32] /
// [E, H, I/32] (MXFP4).  Weight-streaming kernels up to 256 tokens, the
// tiled grouped GEMMs past that.
int run_expert_ffn_q(const moe_dims* d, moe::WFormat fmt, int32_t T, const void* x,
                     const void* guq, const void* gus, const void* dnq, const void* dns,
                     const float* topk_w, const int32_t* offsets, const int32_t* sorted,
                     void* y, void* ws, hipStream_t s) {
  void* h = at<void>(ws, layout(d, T).h);
  const long long H = d->hidden, I = d->expert_inter;
  const bool mx = fmt == moe::WFormat::kMXFP4;
  const long long unit = mx ? 2 : 1;  // weights per stored byte
  const unsigned char* gq = static_cast<const unsigned char*>(guq);
  moe::GateUpArgs g{};
  g.T = T; g.H = d->hidden; g.N = d->expert_inter; g.E = d->num_experts; g.K = d->top_k;
  g.rows = T * d->top_k; g.ident = false; g.bf16 = true;
  g.x = x; g.w_gate = gq; g.w_up = gq + I * H / unit; g.w_stride = 2 * I * H;
  g.offsets = offsets; g.sorted_slots = sorted; g.h = h;
  g.w_fmt = fmt;
  if (mx) {
    g.s_gate = gus;
    g.s_up = static_cast<const unsigned char*>(gus) + I * (H / 32);
    g.s_stride = 2 * I * (H / 32);
  } else {
    g.s_gate = gus;
    g.s_up = static_cast<const float*>(gus) + I;
    g.s_stride = 2 * I;
  }
  hipError_t e = moe::launch_gate_up(g, s);
  if (e != hipSuccess) return hip_fail(e, "expert gate_up (quantized weights)");
  moe::DownArgs dn{};
  dn.T = T; dn.H = d->hidden; dn.N = d->expert_inter; dn.E = d->num_experts; dn.K = d->top_k;
  dn.rows = T * d->top_k; dn.ident = false; dn.bf16 = true;
  dn.y_bf16 = d->slot_dtype == MOE_BF16;
  dn.h = h; dn.w_down = dnq; dn.w_stride = H * I;
  dn.offsets = offsets; dn.sorted_slots = sorted; dn.topk_w = topk_w; dn.y = y;
  dn.w_fmt = fmt; dn.s_down = dns; dn.s_stride = mx ? H * (I / 32) : H;
  e = moe::launch_down(dn, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "expert down (quantized weights)");
}

// MXFP4 kernels stage a block's E8M0 scale rows in LDS, one byte per 32
// weights of a contraction of at most this length.
constexpr int kMaxMxContraction = 8192;

// Format code of the ABI -> the kernels' format, or -1 if unknown.
int wformat_of(int32_t fmt, moe::WFormat& f) {
  switch (fmt) {
    case MOE_W_INT8: f = moe::WFormat::kInt8; return 0;
    case MOE_W_FP8: f = moe::WFormat::kFP8; return 0;
    case MOE_W_MXFP4: f = moe::WFormat::kMXFP4; return 0;
    case MOE_W_MXFP8: f = moe::WFormat::kMXFP8; return 0;
    default: return fail(MOE_ERR_ARG, "weight format %d unknown", fmt);
  }
}

int run_combine(const moe_dims* d, int32_t T, const void* y, const void* addend, void* out,
                hipStream_t s) {
  moe::CombineArgs a{};
  a.T = T; a.H = d->hidden; a.K = d->top_k;
  a.y_bf16 = d->slot_dtype == MOE_BF16; a.act_bf16 = d->act_dtype == MOE_BF16;
  a.y = y; a.addend = addend; a.out = out;
  hipError_t e = moe::launch_combine(a, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_combine");
}

// The matrices of one layer: in the activation dtype (quant == false), or
// codes and scales in format fmt.  Gains, router and layer_scalar are fp32.
struct LayerW {
  const float *g_pre, *g_pre2, *g_post1, *g_post2, *g_post;
  const float *router_w, *router_scale, *per_expert_scale;
  float layer_scalar;
  bool quant;
  moe::WFormat fmt;
  const void *dg, *dgs, *du, *dus, *dd, *dds;  // dense gate, up, down (and scales)
  const void *gu, *gus, *dn, *dns;             // experts' gate_up, down (and scales)
};

// The dense MLP as one group whose rows are the tokens.
void dense_args(const moe_dims* d, int32_t T, const void* x, const void* gate, const void* up,
                const void* down, void* h, void* y, moe::GateUpArgs& g, moe::DownArgs& dd) {
  const bool bf = d->act_dtype == MOE_BF16;
  g.T = T; g.H = d->hidden; g.N = d->dense_inter; g.E = 1; g.K = 1; g.rows = T;
  g.ident = true; g.bf16 = bf; g.x = x; g.w_gate = gate; g.w_up = up;
  g.w_stride = 0; g.offsets = nullptr; g.sorted_slots = nullptr; g.h = h;
  dd.T = T; dd.H = d->hidden; dd.N = d->dense_inter; dd.E = 1; dd.K = 1; dd.rows = T;
  dd.ident = true; dd.bf16 = bf; dd.y_bf16 = d->slot_dtype == MOE_BF16; dd.h = h;
  dd.w_down = down; dd.w_stride = 0; dd.offsets = nullptr; dd.sorted_slots = nullptr;
  dd.topk_w = nullptr; dd.y = y;
}

// One dual-path layer: pre-norms; the dense branch on the side stream; router,
// dispatch and experts on the caller's stream; the epilogue after the join.
int run_layer(const moe_dims* dims, int32_t T, const void* residual, const LayerW& lw,
              void* out, float* ffn_out, int32_t* topk_idx, float* topk_w, void* ws,
              hipStream_t s) {
  int rc;
  const Layout L = layout(dims, T);
  const bool bf = dims->act_dtype == MOE_BF16;
  int32_t* idx = topk_idx ? topk_idx : at<int32_t>(ws, L.idx);
  float* w = topk_w ? topk_w : at<float>(ws, L.w);
  int32_t* counts = at<int32_t>(ws, L.counts);
  int32_t* offsets = at<int32_t>(ws, L.offsets);
  int32_t* sorted = at<int32_t>(ws, L.sorted);
  void* y = at<void>(ws, L.y);
  void* xd = at<void>(ws, L.xd);
  void* xm = at<void>(ws, L.xm);
  void* hd = at<void>(ws, L.hd);
  void* dnb = at<void>(ws, L.dn);

  moe::PreNormArgs pn{};
  pn.T = T; pn.H = dims->hidden; pn.eps = dims->eps; pn.bf16 = bf;
  pn.x = residual; pn.g_pre = lw.g_pre; pn.g_pre2 = lw.g_pre2; pn.xd = xd; pn.xm = xm;
  hipError_t e = moe::launch_prenorm(pn, s);
  if (e != hipSuccess) return hip_fail(e, "ffn layer (prenorm)");

  // dense branch on the side stream, after the pre-norms
  std::lock_guard<std::mutex> lock(g_side_mu);
  SideStream* side = nullptr;
  if ((e = side_stream(side)) != hipSuccess) return hip_fail(e, "ffn layer (side stream)");
  hipStream_t s2 = side->stream;
  if ((e = hipEventRecord(side->fork, s)) != hipSuccess ||
      (e = hipStreamWaitEvent(s2, side->fork, 0)) != hipSuccess)
    return hip_fail(e, "ffn layer (fork)");

  moe::GateUpArgs g{};
  moe::DownArgs dd{};
  dense_args(dims, T, xd, lw.dg, lw.du, lw.dd, hd, dnb, g, dd);
  if (lw.quant) {
    // one group: the per-expert strides are never applied
    g.w_fmt = lw.fmt; g.s_gate = lw.dgs; g.s_up = lw.dus; g.s_stride = 0;
    dd.w_fmt = lw.fmt; dd.s_down = lw.dds; dd.s_stride = 0;
    if ((e = moe::launch_gate_up(g, s2)) != hipSuccess)
      return hip_fail(e, "ffn layer (dense gate_up, quantized weights)");
    if ((e = moe::launch_down(dd, s2)) != hipSuccess)
      return hip_fail(e, "ffn layer (dense down, quantized weights)");
  } else {
    if ((e = moe::launch_gate_up(g, s2)) != hipSuccess)
      return hip_fail(e, "ffn layer (dense gate_up)");
    if ((e = moe::launch_down(dd, s2)) != hipSuccess)
      return hip_fail(e, "ffn layer (dense down)");
  }
  if ((e = hipEventRecord(side->join, s2)) != hipSuccess)
    return hip_fail(e, "ffn layer (join)");

  // router and experts on the caller's stream, meanwhile
  if ((rc = run_router(dims, T, residual, lw.router_w, lw.router_scale, lw.per_expert_scale,
                       lw.g_pre2, idx, w, counts, offsets, sorted, ws, s)))
    return rc;
  rc = lw.quant ? run_expert_ffn_q(dims, lw.fmt, T, xm, lw.gu, lw.gus, lw.dn, lw.dns, w,
                                   offsets, sorted, y, ws, s)
                : run_expert_ffn(dims, T, xm, lw.gu, lw.dn, w, offsets, sorted, y, ws, s);
  if (rc) return rc;
  if ((e = hipStreamWaitEvent(s, side->join, 0)) != hipSuccess)
    return hip_fail(e, "ffn layer (join)");

  moe::EpilogueArgs ep{};
  ep.T = T; ep.H = dims->hidden; ep.K = dims->top_k; ep.eps = dims->eps;
  ep.layer_scalar = lw.layer_scalar; ep.y_bf16 = dims->slot_dtype == MOE_BF16; ep.act_bf16 = bf;
  ep.y = y; ep.dn = dnb; ep.x = residual; ep.g_post1 = lw.g_post1; ep.g_post2 = lw.g_post2;
  ep.g_post = lw.g_post; ep.out = out; ep.ffn_out = ffn_out;
  if ((e = moe::launch_block_epilogue(ep, s)) != hipSuccess)
    return hip_fail(e, "ffn layer (epilogue)");
  return MOE_OK;
}

int check_dense(const moe_dims* d) {
  return d->dense_inter > 0 ? MOE_OK
                            : fail(MOE_ERR_UNSUPPORTED, "the dense MLP needs dense_inter > 0");
}

int check_wgrad(const moe_dims* d, int32_t dt) {
  if (dt != MOE_F32 && dt != MOE_BF16)
    return fail(MOE_ERR_ARG, "d_weights_dtype=%d unknown", dt);
  if (d->act_dtype == MOE_F32 && dt != MOE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "act_dtype F32 requires d_weights_dtype F32");
  return MOE_OK;
}

void set_ffn_grad_ws(moe::FfnGradArgs& a, const FfnGradLayout& L, void* ws) {
  a.ws_row_off = at<unsigned>(ws, L.row_off);
  a.ws_slot_row = at<int32_t>(ws, L.slot_row);
  a.ws_d_gu = at<void>(ws, L.d_gu); a.ws_hw = at<void>(ws, L.hw);
  a.ws_d_xs = at<void>(ws, L.d_xs); a.ws_part = at<float>(ws, L.part);
}

// A caller's list of gradients.
int check_grads(const char* name, int32_t n, const moe_tensor* t) {
  if (n < 0 || n > kMaxGradTensors)
    return fail(MOE_ERR_ARG, "n=%d: need 0..%d", n, kMaxGradTensors);
  if (n > 0 && !t) return fail(MOE_ERR_ARG, "%s is NULL", name);
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].dtype != MOE_F32 && t[i].dtype != MOE_BF16)
      return fail(MOE_ERR_ARG, "%s[%d].dtype=%d unknown", name, i, t[i].dtype);
    if (t[i].numel < 0 || t[i].numel > kMaxGradElements ||
        (total += t[i].numel) > kMaxGradElements)
      return fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^40 elements, or fewer than 0", name);
    if (t[i].numel > 0) {
      if (!t[i].data) return fail(MOE_ERR_ARG, "%s[%d].data is NULL", name, i);
      if (reinterpret_cast<uintptr_t>(t[i].data) % dtype_size(t[i].dtype))
        return fail(MOE_ERR_ARG, "%s[%d].data is not aligned to its type", name, i);
    }
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_workspace_size(const moe_dims* dims, int32_t max_tokens) {
  if (check_dims(dims, true) != MOE_OK) return 0;
  if (check_tokens(dims, max_tokens) != MOE_OK) return 0;
  return layout(dims, max_tokens).total;
}

size_t moe_balance_loss_workspace_size(const moe_dims* dims, int32_t max_tokens) {
  if (check_dims(dims, true) != MOE_OK || check_tokens(dims, max_tokens) != MOE_OK) return 0;
  return balance_layout(dims, max_tokens).total;
}

size_t moe_router_grad_workspace_size(const moe_dims* dims, int32_t max_tokens) {
  if (check_dims(dims, true) != MOE_OK || check_tokens(dims, max_tokens) != MOE_OK) return 0;
  return router_grad_layout(dims, max_tokens).total;
}

size_t moe_expert_ffn_b128_workspace_size(const moe_dims* dims, int32_t max_tokens) {
  if (check_dims(dims, true) != MOE_OK || check_tokens(dims, max_tokens) != MOE_OK) return 0;
  return b128_layout(dims, max_tokens).total;
}

const char* moe_last_error(void) { return g_err.c_str(); }

int moe_router(const moe_dims* dims, int32_t T, const void* x, const float* router_w,
               const float* router_scale, const float* per_expert_scale,
               const float* pre_norm_gain, int32_t* topk_idx, float* topk_w, void* ws,
               size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(router_w); REQUIRE_PTR(router_scale);
  REQUIRE_PTR(per_expert_scale); OPTIONAL_PTR(pre_norm_gain);
  REQUIRE_PTR(topk_idx); REQUIRE_PTR(topk_w);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  return run_router(dims, T, x, router_w, router_scale, per_expert_scale, pre_norm_gain,
                    topk_idx, topk_w, nullptr, nullptr, nullptr, ws,
                    static_cast<hipStream_t>(stream));
}

int moe_route(const moe_dims* dims, int32_t T, const void* x, const float* router_w,
              const float* router_scale, const float* per_expert_scale,
              const float* pre_norm_gain, int32_t* topk_idx, float* topk_w,
              int32_t* expert_counts, int32_t* expert_offsets, int32_t* sorted_slots, void* ws,
              size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(router_w); REQUIRE_PTR(router_scale);
  REQUIRE_PTR(per_expert_scale); OPTIONAL_PTR(pre_norm_gain);
  REQUIRE_PTR(topk_idx); REQUIRE_PTR(topk_w); REQUIRE_PTR(expert_counts);
  REQUIRE_PTR(expert_offsets); REQUIRE_PTR(sorted_slots);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  return run_router(dims, T, x, router_w, router_scale, per_expert_scale, pre_norm_gain,
                    topk_idx, topk_w, expert_counts, expert_offsets, sorted_slots, ws,
                    static_cast<hipStream_t>(stream));
}

int moe_router_logits(const moe_dims* dims, int32_t T, const void* x, const float* router_w,
                      const float* router_scale, const float* per_expert_scale,
                      const float* pre_norm_gain, int32_t* topk_idx, float* topk_w,
                      float* logits, void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(router_w); REQUIRE_PTR(router_scale);
  REQUIRE_PTR(per_expert_scale); OPTIONAL_PTR(pre_norm_gain);
  REQUIRE_PTR(topk_idx); REQUIRE_PTR(topk_w); REQUIRE_PTR(logits);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  return run_router(dims, T, x, router_w, router_scale, per_expert_scale, pre_norm_gain,
                    topk_idx, topk_w, nullptr, nullptr, nullptr, ws,
                    static_cast<hipStream_t>(stream), logits);
}

int moe_balance_loss(const moe_dims* dims, int32_t T, const float* logits,
                     const int32_t* topk_idx, const uint8_t* token_mask, float balance_coef,
                     float z_coef, float* loss, int32_t* expert_counts, float* mean_probs,
                     void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  const auto L = balance_layout(dims, T);
  REQUIRE_PTR(loss); REQUIRE_PTR(expert_counts); REQUIRE_PTR(mean_probs);
  if (T > 0) {
    REQUIRE_PTR(logits); REQUIRE_PTR(topk_idx); OPTIONAL_PTR(token_mask);
    if ((rc = check_ws(L.total, T, ws, ws_bytes))) return rc;
  }
  moe::BalanceArgs a{};
  a.T = T; a.E = dims->num_experts; a.K = dims->top_k;
  a.balance_coef = balance_coef; a.z_coef = z_coef;
  a.logits = logits; a.topk_idx = topk_idx; a.mask = token_mask;
  a.loss = loss; a.counts = expert_counts; a.mean_p = mean_probs;
  a.ws_part_p = at<float>(ws, L.p); a.ws_part_n = at<int32_t>(ws, L.n);
  a.ws_part_z = at<float>(ws, L.z); a.ws_part_live = at<int32_t>(ws, L.live);
  hipError_t e = moe::launch_balance_loss(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_balance_loss");
}

int moe_balance_loss_grad(const moe_dims* dims, int32_t T, const float* logits,
                          const uint8_t* token_mask, const int32_t* expert_counts,
                          const float* loss, float balance_coef, float z_coef,
                          const float* d_loss, float* d_logits, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(logits); OPTIONAL_PTR(token_mask); REQUIRE_PTR(expert_counts); REQUIRE_PTR(loss);
  REQUIRE_PTR(d_loss); REQUIRE_PTR(d_logits);
  moe::BalanceGradArgs a{};
  a.T = T; a.E = dims->num_experts; a.K = dims->top_k;
  a.balance_coef = balance_coef; a.z_coef = z_coef;
  a.logits = logits; a.mask = token_mask; a.counts = expert_counts; a.loss = loss;
  a.d_loss = d_loss; a.d_logits = d_logits;
  hipError_t e = moe::launch_balance_grad(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_balance_loss_grad");
}

int moe_router_grad(const moe_dims* dims, int32_t T, const void* x, const float* router_w,
                    const float* router_scale, const float* per_expert_scale,
                    const float* pre_norm_gain, const float* logits, const int32_t* topk_idx,
                    const uint8_t* token_mask, const float* d_topk_w, const float* d_logits,
                    void* d_x, float* d_router_w, float* d_router_scale,
                    float* d_per_expert_scale, float* d_pre_norm_gain, void* ws,
                    size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  const auto L = router_grad_layout(dims, T);
  REQUIRE_PTR(router_w); REQUIRE_PTR(router_scale); OPTIONAL_PTR(pre_norm_gain);
  REQUIRE_PTR(d_router_w); REQUIRE_PTR(d_router_scale); REQUIRE_PTR(d_per_expert_scale);
  if (pre_norm_gain) {
    REQUIRE_PTR(d_pre_norm_gain);
  } else if (d_pre_norm_gain) {
    return fail(MOE_ERR_ARG, "d_pre_norm_gain without pre_norm_gain");
  }
  if (T > 0) {
    REQUIRE_PTR(x); REQUIRE_PTR(logits); OPTIONAL_PTR(token_mask); OPTIONAL_PTR(d_topk_w);
    OPTIONAL_PTR(d_logits); OPTIONAL_PTR(d_x);
    if (!d_topk_w && !d_logits) return fail(MOE_ERR_ARG, "d_topk_w and d_logits are both NULL");
    if (d_topk_w) {
      REQUIRE_PTR(topk_idx); REQUIRE_PTR(per_expert_scale);
    }
    if ((rc = check_ws(L.total, T, ws, ws_bytes))) return rc;
  }
  moe::RouterGradArgs a{};
  a.T = T; a.H = dims->hidden; a.E = dims->num_experts; a.K = dims->top_k; a.eps = dims->eps;
  a.x_bf16 = dims->act_dtype == MOE_BF16;
  a.x = x; a.router_w = router_w; a.router_scale = router_scale;
  a.per_expert_scale = per_expert_scale; a.pre_gain = pre_norm_gain; a.logits = logits;
  a.topk_idx = topk_idx; a.mask = token_mask; a.d_topk_w = d_topk_w; a.d_logits = d_logits;
  a.d_x = d_x; a.d_router_w = d_router_w; a.d_router_scale = d_router_scale;
  a.d_per_expert_scale = d_per_expert_scale; a.d_pre_gain = d_pre_norm_gain;
  a.ws_dl = at<void>(ws, L.dl); a.ws_beta = at<float>(ws, L.beta);
  a.ws_part_g = at<float>(ws, L.g); a.ws_part_b = at<float>(ws, L.b);
  a.ws_part_pes = at<float>(ws, L.pes);
  hipError_t e = moe::launch_router_grad(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_router_grad");
}

int moe_dispatch(const moe_dims* dims, int32_t T, const int32_t* topk_idx,
                 int32_t* expert_counts, int32_t* expert_offsets, int32_t* sorted_slots,
                 void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(topk_idx); REQUIRE_PTR(expert_counts); REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  return run_dispatch(dims, T, topk_idx, expert_counts, expert_offsets, sorted_slots, ws,
                      static_cast<hipStream_t>(stream));
}

int moe_dense_mask_dispatch(const moe_dims* dims, int32_t T, const int32_t* topk_idx,
                            const float* topk_w, int32_t* expert_offsets, int32_t* sorted_slots,
                            float* w_dense, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if ((long long)T * dims->num_experts > (1 << 20))
    return fail(MOE_ERR_UNSUPPORTED, "T*num_experts=%lld exceeds 2^20",
                (long long)T * dims->num_experts);
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(topk_idx); REQUIRE_PTR(topk_w); REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots); REQUIRE_PTR(w_dense);
  hipError_t e = moe::launch_dense_mask(T, dims->num_experts, dims->top_k, topk_idx, topk_w,
                                        expert_offsets, sorted_slots, w_dense,
                                        static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_dense_mask_dispatch");
}

int moe_expert_ffn(const moe_dims* dims, int32_t T, const void* x, const void* w_gate_up,
                   const void* w_down, const float* topk_w, const int32_t* expert_offsets,
                   const int32_t* sorted_slots, void* y_slots, void* ws, size_t ws_bytes,
                   void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_gate_up); REQUIRE_PTR(w_down); REQUIRE_PTR(topk_w);
  REQUIRE_PTR(expert_offsets); REQUIRE_PTR(sorted_slots); REQUIRE_PTR(y_slots);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  return run_expert_ffn(dims, T, x, w_gate_up, w_down, topk_w, expert_offsets, sorted_slots,
                        y_slots, ws, static_cast<hipStream_t>(stream));
}

int moe_quantize(int32_t fmt, int64_t rows, int32_t cols, const void* w, void* q, void* scale,
                 void* stream) {
  g_err.clear();
  moe::WFormat f;
  if (wformat_of(fmt, f)) return MOE_ERR_ARG;
  if (rows < 0 || rows > (int64_t)1 << 36) return fail(MOE_ERR_ARG, "rows out of range");
  const int align = f == moe::WFormat::kMXFP4 || f == moe::WFormat::kMXFP8 ? 32 : 8;
  if (cols <= 0 || cols % align != 0)
    return fail(MOE_ERR_ARG, "cols must be a positive multiple of %d", align);
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(w); REQUIRE_PTR(q); REQUIRE_PTR(scale);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  switch (f) {
    case moe::WFormat::kMXFP8:
      e = moe::launch_mx8_quantize(rows, cols, w, static_cast<uint8_t*>(q),
                                   static_cast<uint8_t*>(scale), s);
      break;
    case moe::WFormat::kInt8:
      e = moe::launch_quantize_rows(rows, cols, w, static_cast<int8_t*>(q),
                                    static_cast<float*>(scale), s);
      break;
    case moe::WFormat::kFP8:
      e = moe::launch_quantize_fp8(rows, cols, w, static_cast<uint8_t*>(q),
                                   static_cast<float*>(scale), s);
      break;
    default:
      e = moe::launch_quantize_mxfp4(rows, cols, w, static_cast<uint8_t*>(q),
                                     static_cast<uint8_t*>(scale), s);
      break;
  }
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_quantize");
}

int moe_dequantize(int32_t fmt, int64_t rows, int32_t cols, const void* q, const void* scale,
                   float* out, void* stream) {
  g_err.clear();
  moe::WFormat f;
  if (wformat_of(fmt, f)) return MOE_ERR_ARG;
  if (rows < 0 || rows > (int64_t)1 << 36) return fail(MOE_ERR_ARG, "rows out of range");
  const int align = f == moe::WFormat::kMXFP4 || f == moe::WFormat::kMXFP8 ? 32 : 16;
  if (cols <= 0 || cols % align != 0)
    return fail(MOE_ERR_ARG, "cols must be a positive multiple of %d", align);
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(q); REQUIRE_PTR(scale); REQUIRE_PTR(out);
  hipError_t e =
      f == moe::WFormat::kMXFP8
          ? moe::launch_mx8_dequantize(rows, cols, static_cast<const uint8_t*>(q),
                                       static_cast<const uint8_t*>(scale), out,
                                       static_cast<hipStream_t>(stream))
          : moe::launch_dequantize(f, rows, cols, q, scale, out,
                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_dequantize");
}

int moe_expert_ffn_q(const moe_dims* dims, int32_t fmt, int32_t T, const void* x,
                     const void* w_gate_up_q, const void* w_gate_up_scale, const void* w_down_q,
                     const void* w_down_scale, const float* topk_w,
                     const int32_t* expert_offsets, const int32_t* sorted_slots, void* y_slots,
                     void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  moe::WFormat f;
  if (wformat_of(fmt, f)) return MOE_ERR_ARG;
  if (f == moe::WFormat::kMXFP8)
    return fail(MOE_ERR_ARG, "MXFP8 is an activation format, not an expert weight format here");
  if (dims->act_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "quantized experts take bf16 activations");
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_gate_up_q); REQUIRE_PTR(w_gate_up_scale); REQUIRE_PTR(w_down_q);
  REQUIRE_PTR(w_down_scale); REQUIRE_PTR(topk_w); REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots); REQUIRE_PTR(y_slots);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  return run_expert_ffn_q(dims, f, T, x, w_gate_up_q, w_gate_up_scale, w_down_q, w_down_scale,
                          topk_w, expert_offsets, sorted_slots, y_slots, ws,
                          static_cast<hipStream_t>(stream));
}

int moe_expert_ffn_mx(const moe_dims* dims, int32_t fmt, int32_t T, const void* x,
                      const void* w_gate_up_q, const void* w_gate_up_scale, const void* w_down_q,
                      const void* w_down_scale, const float* topk_w,
                      const int32_t* expert_offsets, const int32_t* sorted_slots, void* y_slots,
                      void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  moe::WFormat f;
  if (wformat_of(fmt, f)) return MOE_ERR_ARG;
  if (f != moe::WFormat::kFP8 && f != moe::WFormat::kMXFP4)
    return fail(MOE_ERR_ARG, "moe_expert_ffn_mx takes E4M3 or MXFP4 expert weights");
  if (dims->act_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "8-bit / 4-bit experts take bf16 activations");
  if (!moe::mx_uses_stream_kernels(T, T * dims->top_k, dims->num_experts) &&
      !moe::mx_tiled_supported(dims->hidden, dims->expert_inter))
    return fail(MOE_ERR_UNSUPPORTED, "8-bit / 4-bit experts past 256 tokens: hidden and "
                                     "expert_inter must be multiples of 64, at most 4096");
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_gate_up_q); REQUIRE_PTR(w_gate_up_scale); REQUIRE_PTR(w_down_q);
  REQUIRE_PTR(w_down_scale); REQUIRE_PTR(topk_w); REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots); REQUIRE_PTR(y_slots);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  const Layout L = layout(dims, T);
  moe::MxArgs a{};
  a.T = T; a.H = dims->hidden; a.I = dims->expert_inter; a.E = dims->num_experts;
  a.K = dims->top_k; a.rows = T * dims->top_k; a.fmt = f;
  a.y_bf16 = dims->slot_dtype == MOE_BF16;
  a.x = x; a.xq = at<uint8_t>(ws, L.xq); a.xs = at<uint8_t>(ws, L.xs);
  a.hq = at<uint8_t>(ws, L.hq); a.hs = at<uint8_t>(ws, L.hs);
  a.gate_up_q = w_gate_up_q; a.gate_up_s = w_gate_up_scale;
  a.down_q = w_down_q; a.down_s = w_down_scale;
  a.offsets = expert_offsets; a.sorted_slots = sorted_slots; a.topk_w = topk_w; a.y = y_slots;
  hipError_t e = moe::launch_expert_ffn_mx(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_mx");
}

namespace {

// Shape of a block-scaled matrix batch.
int check_b128(int32_t block_rows, int64_t batch, int32_t rows, int32_t cols) {
  if (block_rows != 1 && block_rows != 128)
    return fail(MOE_ERR_ARG, "block_rows=%d: need 1 or 128", block_rows);
  if (batch < 0 || rows < 0 || batch > (int64_t)1 << 31 || rows > 1 << 21)
    return fail(MOE_ERR_ARG, "batch or rows out of range");
  if (cols < 16 || cols > 65536 || cols % 16)
    return fail(MOE_ERR_ARG, "cols=%d: need a multiple of 16 in [16, 65536]", cols);
  // a launch counts its lanes in 32 bits: 16 for the 128 values that share a scale
  if (batch * rows >= ((int64_t)1 << 28) / ((cols + 127) / 128))
    return fail(MOE_ERR_UNSUPPORTED, "2^28 or more pieces of 128 values");
  return MOE_OK;
}

int check_linear(int32_t T, int32_t out_features, int32_t in_features) {
  if (T < 0 || T > 65536) return fail(MOE_ERR_ARG, "T=%d: need 0..65536", T);
  if (out_features < 1 || out_features > 1 << 18)
    return fail(MOE_ERR_UNSUPPORTED, "out_features=%d: need 1..262144", out_features);
  if (in_features < 16 || in_features > 16384 || in_features % 16)
    return fail(MOE_ERR_UNSUPPORTED, "in_features=%d: need a multiple of 16 in [16, 16384]",
                in_features);
  return MOE_OK;
}

size_t linear_scale_offset(int32_t T, int32_t in_features) {
  return align256((size_t)T * ((in_features + 127) / 128 * 128));
}

}  // namespace

int moe_quantize_b128(int32_t block_rows, int64_t batch, int32_t rows, int32_t cols,
                      const void* w, uint8_t* q, float* scale, void* stream) {
  int rc;
  if ((rc = check_b128(block_rows, batch, rows, cols))) return rc;
  g_err.clear();
  if (batch == 0 || rows == 0) return MOE_OK;
  REQUIRE_PTR(w); REQUIRE_PTR(q); REQUIRE_PTR(scale);
  hipError_t e = moe::launch_quantize_b128(block_rows, batch, rows, cols, w, q, scale,
                                           static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_quantize_b128");
}

int moe_dequantize_b128(int32_t block_rows, int64_t batch, int32_t rows, int32_t cols,
                        const uint8_t* q, const float* scale, float* out, void* stream) {
  int rc;
  if ((rc = check_b128(block_rows, batch, rows, cols))) return rc;
  g_err.clear();
  if (batch == 0 || rows == 0) return MOE_OK;
  REQUIRE_PTR(q); REQUIRE_PTR(scale); REQUIRE_PTR(out);
  hipError_t e = moe::launch_dequantize_b128(block_rows, batch, rows, cols, q, scale, out,
                                             static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_dequantize_b128");
}

size_t moe_linear_b128_workspace_size(int32_t max_tokens, int32_t in_features) {
  if (check_linear(max_tokens, 1, in_features) != MOE_OK) return 0;
  return linear_scale_offset(max_tokens, in_features) +
         align256(4 * (size_t)max_tokens * ((in_features + 127) / 128)) + 256;
}

int moe_linear_b128(int32_t T, int32_t out_features, int32_t in_features, const void* x,
                    const uint8_t* w_q, const float* w_scale, void* y, int32_t y_dtype, void* ws,
                    size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_linear(T, out_features, in_features))) return rc;
  if (y_dtype != MOE_F32 && y_dtype != MOE_BF16)
    return fail(MOE_ERR_ARG, "y_dtype=%d unknown", y_dtype);
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_q); REQUIRE_PTR(w_scale); REQUIRE_PTR(y);
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(MOE_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  const size_t need = moe_linear_b128_workspace_size(T, in_features);
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed for T=%d", ws_bytes, need,
                T);
  moe::B128Args a{};
  a.T = T; a.rows = T; a.E = 1; a.K = 1; a.Kd = in_features; a.N = out_features; a.ident = true;
  uint8_t* xq = at<uint8_t>(ws, 0);
  float* xs = at<float>(ws, linear_scale_offset(T, in_features));
  a.xq = xq; a.xscale = xs; a.wq = w_q; a.wscale = w_scale; a.y = y;
  hipError_t e = moe::launch_linear_b128(a, x, xq, xs, y_dtype == MOE_BF16,
                                         static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_linear_b128");
}

int moe_expert_ffn_b128(const moe_dims* dims, int32_t T, const void* x,
                        const uint8_t* w_gate_up_q, const float* w_gate_up_scale,
                        const uint8_t* w_down_q, const float* w_down_scale, const float* topk_w,
                        const int32_t* expert_offsets, const int32_t* sorted_slots,
                        void* y_slots, void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  const auto L = b128_layout(dims, T);
  if (dims->act_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "block-scaled E4M3 experts take bf16 activations");
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_gate_up_q); REQUIRE_PTR(w_gate_up_scale); REQUIRE_PTR(w_down_q);
  REQUIRE_PTR(w_down_scale); REQUIRE_PTR(topk_w); REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots); REQUIRE_PTR(y_slots);
  if ((rc = check_ws(L.total, T, ws, ws_bytes))) return rc;
  moe::B128Args gu{};
  gu.T = T; gu.rows = T * dims->top_k; gu.E = dims->num_experts; gu.K = dims->top_k;
  gu.offsets = expert_offsets; gu.sorted_slots = sorted_slots; gu.topk_w = topk_w;
  moe::B128Args dn = gu;
  gu.Kd = dims->hidden; gu.N = dims->expert_inter;
  gu.xq = at<uint8_t>(ws, L.xq); gu.xscale = at<float>(ws, L.xs);
  gu.wq = w_gate_up_q; gu.wscale = w_gate_up_scale;
  gu.h = at<float>(ws, L.h); gu.hq = at<uint8_t>(ws, L.hq); gu.hscale = at<float>(ws, L.hs);
  dn.Kd = dims->expert_inter; dn.N = dims->hidden;
  dn.xq = gu.hq; dn.xscale = gu.hscale; dn.wq = w_down_q; dn.wscale = w_down_scale;
  dn.y = y_slots;
  hipError_t e = moe::launch_expert_ffn_b128(gu, dn, x, at<uint8_t>(ws, L.xq),
                                             at<float>(ws, L.xs),
                                             dims->slot_dtype == MOE_BF16,
                                             static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_b128");
}

int moe_quantize_int8(int64_t rows, int32_t cols, const void* w, int8_t* q, float* scale,
                      void* stream) {
  return moe_quantize(MOE_W_INT8, rows, cols, w, q, scale, stream);
}

int moe_expert_ffn_int8(const moe_dims* dims, int32_t T, const void* x, const int8_t* w_gate_up_q,
                        const float* w_gate_up_scale, const int8_t* w_down_q,
                        const float* w_down_scale, const float* topk_w,
                        const int32_t* expert_offsets, const int32_t* sorted_slots, void* y_slots,
                        void* ws, size_t ws_bytes, void* stream) {
  return moe_expert_ffn_q(dims, MOE_W_INT8, T, x, w_gate_up_q, w_gate_up_scale, w_down_q,
                          w_down_scale, topk_w, expert_offsets, sorted_slots, y_slots, ws,
                          ws_bytes, stream);
}

int moe_expert_gate_up(const moe_dims* dims, int32_t T, const void* x, const void* w_gate_up,
                       const int32_t* expert_offsets, const int32_t* sorted_slots, void* h,
                       void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_gate_up); REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots); REQUIRE_PTR(h);
  return run_gate_up(dims, T, x, w_gate_up, expert_offsets, sorted_slots, h,
                     static_cast<hipStream_t>(stream));
}

int moe_expert_gate_up_timed(const moe_dims* dims, int32_t T, const void* x,
                             const void* w_gate_up, const int32_t* expert_offsets,
                             const int32_t* sorted_slots, void* h, void* stream,
                             void* start_event, void* stop_event) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (!start_event || !stop_event) return fail(MOE_ERR_ARG, "start_event and stop_event are required");
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_gate_up); REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots); REQUIRE_PTR(h);
  return run_gate_up(dims, T, x, w_gate_up, expert_offsets, sorted_slots, h,
                     static_cast<hipStream_t>(stream), static_cast<hipEvent_t>(start_event),
                     static_cast<hipEvent_t>(stop_event));
}

int moe_expert_down(const moe_dims* dims, int32_t T, const void* h, const void* w_down,
                    const float* topk_w, const int32_t* expert_offsets,
                    const int32_t* sorted_slots, void* y_slots, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(h); REQUIRE_PTR(w_down); REQUIRE_PTR(topk_w); REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots); REQUIRE_PTR(y_slots);
  return run_down(dims, T, h, w_down, topk_w, expert_offsets, sorted_slots, y_slots,
                  static_cast<hipStream_t>(stream));
}

int moe_combine(const moe_dims* dims, int32_t T, const void* y_slots, const void* addend,
                void* out, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(y_slots); OPTIONAL_PTR(addend); REQUIRE_PTR(out);
  return run_combine(dims, T, y_slots, addend, out, static_cast<hipStream_t>(stream));
}

int moe_forward(const moe_dims* dims, int32_t T, const void* x, const float* router_w,
                const float* router_scale, const float* per_expert_scale,
                const void* w_gate_up, const void* w_down, void* out, int32_t* topk_idx,
                float* topk_w, void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(router_w); REQUIRE_PTR(router_scale);
  REQUIRE_PTR(per_expert_scale); REQUIRE_PTR(w_gate_up); REQUIRE_PTR(w_down); REQUIRE_PTR(out);
  OPTIONAL_PTR(topk_idx); OPTIONAL_PTR(topk_w);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  return run_forward(dims, T, x, router_w, router_scale, per_expert_scale, w_gate_up, w_down,
                     out, topk_idx, topk_w, ws, static_cast<hipStream_t>(stream));
}

int moe_forward_noalloc(const moe_dims* dims, int32_t T, const void* x, const float* router_w,
                        const float* router_scale, const float* per_expert_scale,
                        const void* w_gate_up, const void* w_down, void* out, int32_t* topk_idx,
                        float* topk_w, void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(router_w); REQUIRE_PTR(router_scale);
  REQUIRE_PTR(per_expert_scale); REQUIRE_PTR(w_gate_up); REQUIRE_PTR(w_down); REQUIRE_PTR(out);
  OPTIONAL_PTR(topk_idx); OPTIONAL_PTR(topk_w);
  const size_t need = layout(dims, T).base_end;  // moe_forward uses no MXFP8 region
  if (need > kNoAllocScratchBytes)
    return fail(MOE_ERR_WORKSPACE,
                "moe_forward_noalloc: T=%d needs %zu bytes of scratch, the library's array "
                "holds %zu",
                T, need, kNoAllocScratchBytes);
  void* ws = nullptr;
  hipError_t e = noalloc_scratch(ws);
  if (e != hipSuccess) return hip_fail(e, "moe_forward_noalloc (scratch address)");
  return run_forward(dims, T, x, router_w, router_scale, per_expert_scale, w_gate_up, w_down,
                     out, topk_idx, topk_w, ws, static_cast<hipStream_t>(stream));
}

}  // extern "C"

namespace {

int run_forward(const moe_dims* dims, int32_t T, const void* x, const float* router_w,
                const float* router_scale, const float* per_expert_scale,
                const void* w_gate_up, const void* w_down, void* out, int32_t* topk_idx,
                float* topk_w, void* ws, hipStream_t s) {
  int rc;
  const Layout L = layout(dims, T);
  int32_t* idx = topk_idx ? topk_idx : at<int32_t>(ws, L.idx);
  float* w = topk_w ? topk_w : at<float>(ws, L.w);
  int32_t* counts = at<int32_t>(ws, L.counts);
  int32_t* offsets = at<int32_t>(ws, L.offsets);
  int32_t* sorted = at<int32_t>(ws, L.sorted);
  void* y = at<void>(ws, L.y);
  if ((rc = run_router(dims, T, x, router_w, router_scale, per_expert_scale, nullptr, idx, w,
                       counts, offsets, sorted, ws, s)))
    return rc;
  if ((rc = run_expert_ffn(dims, T, x, w_gate_up, w_down, w, offsets, sorted, y, ws, s)))
    return rc;
  return run_combine(dims, T, y, nullptr, out, s);
}

}  // namespace

extern "C" {

int gemma4_ffn_block(const moe_dims* dims, int32_t T, const void* residual,
                     const gemma4_ffn_weights* wt, void* out, float* ffn_out,
                     int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                     void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  if (dims->dense_inter <= 0)
    return fail(MOE_ERR_UNSUPPORTED, "gemma4_ffn_block needs dense_inter > 0");
  g_err.clear();
  if (T == 0) return MOE_OK;
  if (!wt) return fail(MOE_ERR_ARG, "weights is NULL");
  REQUIRE_PTR(residual); REQUIRE_PTR(out); OPTIONAL_PTR(ffn_out);
  OPTIONAL_PTR(topk_idx); OPTIONAL_PTR(topk_w);
  REQUIRE_PTR(wt->g_pre); REQUIRE_PTR(wt->g_pre2); REQUIRE_PTR(wt->g_post1);
  REQUIRE_PTR(wt->g_post2); REQUIRE_PTR(wt->g_post);
  REQUIRE_PTR(wt->dense_gate); REQUIRE_PTR(wt->dense_up); REQUIRE_PTR(wt->dense_down);
  REQUIRE_PTR(wt->router_w); REQUIRE_PTR(wt->router_scale); REQUIRE_PTR(wt->per_expert_scale);
  REQUIRE_PTR(wt->w_gate_up); REQUIRE_PTR(wt->w_down);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  LayerW lw{};
  lw.g_pre = wt->g_pre; lw.g_pre2 = wt->g_pre2; lw.g_post1 = wt->g_post1;
  lw.g_post2 = wt->g_post2; lw.g_post = wt->g_post;
  lw.router_w = wt->router_w; lw.router_scale = wt->router_scale;
  lw.per_expert_scale = wt->per_expert_scale; lw.layer_scalar = wt->layer_scalar;
  lw.quant = false;
  lw.dg = wt->dense_gate; lw.du = wt->dense_up; lw.dd = wt->dense_down;
  lw.gu = wt->w_gate_up; lw.dn = wt->w_down;
  return run_layer(dims, T, residual, lw, out, ffn_out, topk_idx, topk_w, ws,
                   static_cast<hipStream_t>(stream));
}

int gemma4_ffn_block_q(const moe_dims* dims, int32_t T, const void* residual,
                       const gemma4_ffn_weights_q* wt, void* out, float* ffn_out,
                       int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                       void* stream) {
  int rc;
  if ((rc = check_dims(dims)) || (rc = check_tokens(dims, T))) return rc;
  if (dims->dense_inter <= 0)
    return fail(MOE_ERR_UNSUPPORTED, "gemma4_ffn_block_q needs dense_inter > 0");
  if (dims->act_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "quantized layer takes bf16 activations");
  g_err.clear();
  if (T == 0) return MOE_OK;
  if (!wt) return fail(MOE_ERR_ARG, "weights is NULL");
  moe::WFormat f;
  if (wformat_of(wt->fmt, f)) return MOE_ERR_ARG;
  if (f == moe::WFormat::kMXFP8)
    return fail(MOE_ERR_ARG, "MXFP8 is an activation format, not a weight format here");
  if (f == moe::WFormat::kMXFP4 && dims->dense_inter > kMaxMxContraction)
    return fail(MOE_ERR_UNSUPPORTED, "MXFP4 weights: dense_inter=%d exceeds %d",
                dims->dense_inter, kMaxMxContraction);
  REQUIRE_PTR(residual); REQUIRE_PTR(out); OPTIONAL_PTR(ffn_out);
  OPTIONAL_PTR(topk_idx); OPTIONAL_PTR(topk_w);
  REQUIRE_PTR(wt->g_pre); REQUIRE_PTR(wt->g_pre2); REQUIRE_PTR(wt->g_post1);
  REQUIRE_PTR(wt->g_post2); REQUIRE_PTR(wt->g_post);
  REQUIRE_PTR(wt->dense_gate_q); REQUIRE_PTR(wt->dense_gate_scale);
  REQUIRE_PTR(wt->dense_up_q); REQUIRE_PTR(wt->dense_up_scale);
  REQUIRE_PTR(wt->dense_down_q); REQUIRE_PTR(wt->dense_down_scale);
  REQUIRE_PTR(wt->router_w); REQUIRE_PTR(wt->router_scale); REQUIRE_PTR(wt->per_expert_scale);
  REQUIRE_PTR(wt->gate_up_q); REQUIRE_PTR(wt->gate_up_scale);
  REQUIRE_PTR(wt->down_q); REQUIRE_PTR(wt->down_scale);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  LayerW lw{};
  lw.g_pre = wt->g_pre; lw.g_pre2 = wt->g_pre2; lw.g_post1 = wt->g_post1;
  lw.g_post2 = wt->g_post2; lw.g_post = wt->g_post;
  lw.router_w = wt->router_w; lw.router_scale = wt->router_scale;
  lw.per_expert_scale = wt->per_expert_scale; lw.layer_scalar = wt->layer_scalar;
  lw.quant = true; lw.fmt = f;
  lw.dg = wt->dense_gate_q; lw.dgs = wt->dense_gate_scale;
  lw.du = wt->dense_up_q; lw.dus = wt->dense_up_scale;
  lw.dd = wt->dense_down_q; lw.dds = wt->dense_down_scale;
  lw.gu = wt->gate_up_q; lw.gus = wt->gate_up_scale;
  lw.dn = wt->down_q; lw.dns = wt->down_scale;
  return run_layer(dims, T, residual, lw, out, ffn_out, topk_idx, topk_w, ws,
                   static_cast<hipStream_t>(stream));
}

// ---- the rest of the layer's training step ---------------------------------

int moe_expert_ffn_keep(const moe_dims* dims, int32_t T, const void* x, const void* w_gate_up,
                        const void* w_down, const float* topk_w, const int32_t* expert_offsets,
                        const int32_t* sorted_slots, void* gate_up, void* y_slots, void* ws,
                        size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_gate_up); REQUIRE_PTR(w_down); REQUIRE_PTR(topk_w);
  REQUIRE_PTR(expert_offsets); REQUIRE_PTR(sorted_slots); REQUIRE_PTR(gate_up);
  REQUIRE_PTR(y_slots);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  return run_expert_ffn(dims, T, x, w_gate_up, w_down, topk_w, expert_offsets, sorted_slots,
                        y_slots, ws, static_cast<hipStream_t>(stream), gate_up);
}

size_t moe_expert_ffn_grad_workspace_size(const moe_dims* dims, int32_t max_tokens) {
  if (check_dims(dims, true) != MOE_OK || check_tokens(dims, max_tokens) != MOE_OK) return 0;
  return ffn_grad_layout(dims, (long long)max_tokens * dims->top_k, dims->expert_inter, true)
      .total;
}

int moe_expert_ffn_grad(const moe_dims* dims, int32_t T, const void* x, const void* w_gate_up,
                        const void* w_down, const float* topk_w, const int32_t* expert_offsets,
                        const int32_t* sorted_slots, const void* gate_up,
                        const uint8_t* token_mask, const void* d_out, void* d_x, float* d_topk_w,
                        int32_t d_weights_dtype, void* d_w_gate_up, void* d_w_down, void* ws,
                        size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T)) ||
      (rc = check_wgrad(dims, d_weights_dtype)))
    return rc;
  g_err.clear();
  OPTIONAL_PTR(d_x); OPTIONAL_PTR(d_topk_w); OPTIONAL_PTR(d_w_gate_up); OPTIONAL_PTR(d_w_down);
  if (!d_x && !d_topk_w && !d_w_gate_up && !d_w_down)
    return fail(MOE_ERR_ARG, "every output is NULL");
  const long long H = dims->hidden, I = dims->expert_inter;
  const FfnGradLayout L = ffn_grad_layout(dims, (long long)T * dims->top_k, I, true);
  if (T > 0) {
    REQUIRE_PTR(x); REQUIRE_PTR(w_gate_up); REQUIRE_PTR(w_down); REQUIRE_PTR(topk_w);
    REQUIRE_PTR(expert_offsets); REQUIRE_PTR(sorted_slots); REQUIRE_PTR(gate_up);
    OPTIONAL_PTR(token_mask); REQUIRE_PTR(d_out);
    if ((rc = check_ws(L.total, T, ws, ws_bytes))) return rc;
  }
  const size_t act = dtype_size(dims->act_dtype), wg = dtype_size(d_weights_dtype);
  moe::FfnGradArgs a{};
  a.T = T; a.H = dims->hidden; a.I = dims->expert_inter; a.E = dims->num_experts;
  a.K = dims->top_k; a.rows = T * dims->top_k; a.ident = false;
  a.bf16 = dims->act_dtype == MOE_BF16; a.wgrad_bf16 = d_weights_dtype == MOE_BF16;
  a.xs_bf16 = dims->slot_dtype == MOE_BF16;
  a.x = x; a.w_gate = w_gate_up;
  a.w_up = w_gate_up ? static_cast<const char*>(w_gate_up) + act * I * H : nullptr;
  a.gu_stride = 2 * I * H; a.w_down = w_down; a.dn_stride = H * I;
  a.topk_w = topk_w; a.offsets = expert_offsets; a.sorted_slots = sorted_slots;
  a.kept = gate_up; a.mask = token_mask; a.d_out = d_out; a.d_x = d_x; a.d_topk_w = d_topk_w;
  a.d_gate = d_w_gate_up;
  a.d_up = d_w_gate_up ? static_cast<char*>(d_w_gate_up) + wg * I * H : nullptr;
  a.d_down = d_w_down;
  set_ffn_grad_ws(a, L, ws);
  hipError_t e = moe::launch_ffn_grad(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_grad");
}

int gemma4_dense_mlp(const moe_dims* dims, int32_t T, const void* x, const void* dense_gate,
                     const void* dense_up, const void* dense_down, void* gate_up, void* y,
                     void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T)) || (rc = check_dense(dims)))
    return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(dense_gate); REQUIRE_PTR(dense_up); REQUIRE_PTR(dense_down);
  OPTIONAL_PTR(gate_up); REQUIRE_PTR(y);
  if ((rc = check_ws(dims, T, ws, ws_bytes))) return rc;
  moe::GateUpArgs g{};
  moe::DownArgs dd{};
  dense_args(dims, T, x, dense_gate, dense_up, dense_down, at<void>(ws, layout(dims, T).hd), y, g,
             dd);
  g.keep = gate_up;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = moe::launch_gate_up(g, s);
  if (e == hipSuccess) e = moe::launch_down(dd, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "gemma4_dense_mlp");
}

size_t gemma4_dense_mlp_grad_workspace_size(const moe_dims* dims, int32_t max_tokens) {
  if (check_dims(dims, true) != MOE_OK || check_tokens(dims, max_tokens) != MOE_OK ||
      check_dense(dims) != MOE_OK)
    return 0;
  return ffn_grad_layout(dims, max_tokens, dims->dense_inter, false).total;
}

int gemma4_dense_mlp_grad(const moe_dims* dims, int32_t T, const void* x, const void* dense_gate,
                          const void* dense_up, const void* dense_down, const void* gate_up,
                          const uint8_t* token_mask, const void* d_y, void* d_x,
                          int32_t d_weights_dtype, void* d_gate, void* d_up, void* d_down,
                          void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T)) || (rc = check_dense(dims)) ||
      (rc = check_wgrad(dims, d_weights_dtype)))
    return rc;
  g_err.clear();
  OPTIONAL_PTR(d_x); OPTIONAL_PTR(d_gate); OPTIONAL_PTR(d_up); OPTIONAL_PTR(d_down);
  if (!d_gate != !d_up) return fail(MOE_ERR_ARG, "d_gate and d_up go together");
  if (!d_x && !d_gate && !d_down) return fail(MOE_ERR_ARG, "every output is NULL");
  const FfnGradLayout L = ffn_grad_layout(dims, T, dims->dense_inter, false);
  if (T > 0) {
    REQUIRE_PTR(x); REQUIRE_PTR(dense_gate); REQUIRE_PTR(dense_up); REQUIRE_PTR(dense_down);
    REQUIRE_PTR(gate_up); OPTIONAL_PTR(token_mask); REQUIRE_PTR(d_y);
    if ((rc = check_ws(L.total, T, ws, ws_bytes))) return rc;
  }
  moe::FfnGradArgs a{};
  a.T = T; a.H = dims->hidden; a.I = dims->dense_inter; a.E = 1; a.K = 1; a.rows = T;
  a.ident = true; a.bf16 = dims->act_dtype == MOE_BF16;
  a.wgrad_bf16 = d_weights_dtype == MOE_BF16;
  a.x = x; a.w_gate = dense_gate; a.w_up = dense_up; a.w_down = dense_down;
  a.kept = gate_up; a.mask = token_mask; a.d_out = d_y; a.d_x = d_x;
  a.d_gate = d_gate; a.d_up = d_up; a.d_down = d_down;
  set_ffn_grad_ws(a, L, ws);
  hipError_t e = moe::launch_ffn_grad(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "gemma4_dense_mlp_grad");
}

int gemma4_pre_norms(const moe_dims* dims, int32_t T, const void* x, const float* g_pre,
                     const float* g_pre2, void* xd, void* xm, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(g_pre); REQUIRE_PTR(g_pre2); REQUIRE_PTR(xd); REQUIRE_PTR(xm);
  moe::PreNormArgs a{};
  a.T = T; a.H = dims->hidden; a.eps = dims->eps; a.bf16 = dims->act_dtype == MOE_BF16;
  a.x = x; a.g_pre = g_pre; a.g_pre2 = g_pre2; a.xd = xd; a.xm = xm;
  hipError_t e = moe::launch_prenorm(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "gemma4_pre_norms");
}

int gemma4_post_norms(const moe_dims* dims, int32_t T, const void* x, const void* y_slots,
                      const void* dn, const float* g_post1, const float* g_post2,
                      const float* g_post, float layer_scalar, void* out, void* moe_sum,
                      float* ffn_out, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(y_slots); REQUIRE_PTR(dn); REQUIRE_PTR(g_post1);
  REQUIRE_PTR(g_post2); REQUIRE_PTR(g_post); REQUIRE_PTR(out); OPTIONAL_PTR(moe_sum);
  OPTIONAL_PTR(ffn_out);
  moe::EpilogueArgs a{};
  a.T = T; a.H = dims->hidden; a.K = dims->top_k; a.eps = dims->eps;
  a.layer_scalar = layer_scalar; a.y_bf16 = dims->slot_dtype == MOE_BF16;
  a.act_bf16 = dims->act_dtype == MOE_BF16; a.y = y_slots; a.dn = dn; a.x = x;
  a.g_post1 = g_post1; a.g_post2 = g_post2; a.g_post = g_post; a.out = out; a.ffn_out = ffn_out;
  a.moe_sum = moe_sum;
  hipError_t e = moe::launch_block_epilogue(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "gemma4_post_norms");
}

size_t gemma4_norms_grad_workspace_size(const moe_dims* dims, int32_t max_tokens) {
  if (check_dims(dims, true) != MOE_OK || check_tokens(dims, max_tokens) != MOE_OK) return 0;
  return norms_grad_layout(dims, max_tokens).total;
}

int gemma4_pre_norms_grad(const moe_dims* dims, int32_t T, const void* x, const float* g_pre,
                          const float* g_pre2, const uint8_t* token_mask, const void* d_xd,
                          const void* d_xm, const void* d_x_add, const void* d_out,
                          float layer_scalar, void* d_x, float* d_g_pre, float* d_g_pre2,
                          void* ws, size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  REQUIRE_PTR(d_g_pre); REQUIRE_PTR(d_g_pre2);
  const NormsGradLayout L = norms_grad_layout(dims, T);
  if (T > 0) {
    REQUIRE_PTR(x); REQUIRE_PTR(g_pre); REQUIRE_PTR(g_pre2); OPTIONAL_PTR(token_mask);
    REQUIRE_PTR(d_xd); REQUIRE_PTR(d_xm); OPTIONAL_PTR(d_x_add); OPTIONAL_PTR(d_out);
    REQUIRE_PTR(d_x);
    if ((rc = check_ws(L.total, T, ws, ws_bytes))) return rc;
  }
  moe::PreNormGradArgs a{};
  a.T = T; a.H = dims->hidden; a.eps = dims->eps; a.scalar = layer_scalar;
  a.bf16 = dims->act_dtype == MOE_BF16;
  a.x = x; a.g1 = g_pre; a.g2 = g_pre2; a.mask = token_mask; a.d_xd = d_xd; a.d_xm = d_xm;
  a.d_add = d_x_add; a.d_out = d_out; a.d_x = d_x; a.d_g1 = d_g_pre; a.d_g2 = d_g_pre2;
  a.ws_part = at<float>(ws, L.part);
  hipError_t e = moe::launch_pre_norms_grad(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "gemma4_pre_norms_grad");
}

int gemma4_post_norms_grad(const moe_dims* dims, int32_t T, const void* x, const void* dn,
                           const void* moe_sum, const float* g_post1, const float* g_post2,
                           const float* g_post, float layer_scalar, const uint8_t* token_mask,
                           const void* d_out, void* d_dn, void* d_moe, float* d_g_post1,
                           float* d_g_post2, float* d_g_post, float* d_layer_scalar, void* ws,
                           size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(dims, true)) || (rc = check_tokens(dims, T))) return rc;
  g_err.clear();
  REQUIRE_PTR(d_g_post1); REQUIRE_PTR(d_g_post2); REQUIRE_PTR(d_g_post);
  OPTIONAL_PTR(d_layer_scalar);
  const NormsGradLayout L = norms_grad_layout(dims, T);
  if (T > 0) {
    if (d_layer_scalar) REQUIRE_PTR(x);
    REQUIRE_PTR(dn); REQUIRE_PTR(moe_sum); REQUIRE_PTR(g_post1); REQUIRE_PTR(g_post2);
    REQUIRE_PTR(g_post); OPTIONAL_PTR(token_mask); REQUIRE_PTR(d_out); REQUIRE_PTR(d_dn);
    REQUIRE_PTR(d_moe);
    if ((rc = check_ws(L.total, T, ws, ws_bytes))) return rc;
  }
  moe::PostNormGradArgs a{};
  a.T = T; a.H = dims->hidden; a.eps = dims->eps; a.scalar = layer_scalar;
  a.bf16 = dims->act_dtype == MOE_BF16; a.y_bf16 = dims->slot_dtype == MOE_BF16;
  a.x = x; a.dn = dn; a.moe_sum = moe_sum; a.g1 = g_post1; a.g2 = g_post2; a.g3 = g_post;
  a.mask = token_mask; a.d_out = d_out; a.d_dn = d_dn; a.d_moe = d_moe;
  a.d_g1 = d_g_post1; a.d_g2 = d_g_post2; a.d_g3 = d_g_post; a.d_scalar = d_layer_scalar;
  a.ws_part = at<float>(ws, L.part); a.ws_scalar = at<double>(ws, L.scalar);
  hipError_t e = moe::launch_post_norms_grad(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "gemma4_post_norms_grad");
}

size_t moe_grad_norm_workspace_size(int32_t n, const moe_tensor* grads) {
  if (check_grads("grads", n, grads) != MOE_OK) return 0;
  return align256(8 * (size_t)moe::grad_norm_parts(n, grads)) + 256;
}

int moe_grad_norm(int32_t n, const moe_tensor* grads, float max_norm, float* norm, void* ws,
                  size_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_grads("grads", n, grads))) return rc;
  if (!(max_norm > 0.0f)) return fail(MOE_ERR_ARG, "max_norm must be > 0");
  g_err.clear();
  REQUIRE_PTR(norm);
  const size_t need = align256(8 * (size_t)moe::grad_norm_parts(n, grads)) + 256;
  if ((rc = check_ws(need, "this list", ws, ws_bytes))) return rc;
  hipError_t e = moe::launch_grad_norm(n, grads, max_norm, norm, static_cast<double*>(ws),
                                       static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_grad_norm");
}

int moe_grad_clip(int32_t n, const moe_tensor* grads, const float* norm, const moe_tensor* out,
                  void* stream) {
  int rc;
  if ((rc = check_grads("grads", n, grads)) || (out && (rc = check_grads("out", n, out))))
    return rc;
  for (int32_t i = 0; out && i < n; ++i)
    if (grads[i].numel != out[i].numel)
      return fail(MOE_ERR_ARG, "out[%d] has %lld elements, grads[%d] %lld", i,
                  (long long)out[i].numel, i, (long long)grads[i].numel);
  g_err.clear();
  if (n == 0) return MOE_OK;
  REQUIRE_PTR(norm);
  hipError_t e = moe::launch_grad_clip(n, grads, norm, out, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_grad_clip");
}

}  // extern "C"
