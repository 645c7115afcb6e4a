// C ABI of the MoE layer library: argument validation, workspace layout and the launch sequence
// of each call.  Every call validates everything on the host before it enqueues anything, then
// enqueues its kernels on the caller's stream without synchronising.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <memory>
#include <mutex>
#include <new>
#include <string>

#include "../../include/moe.h"
#include "internal.h"
#include "philox.h"
#include "w4.h"

using namespace moe;

namespace {

thread_local std::string g_err;

moe_status fail(moe_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

moe_status hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return MOE_OK;
  return fail(MOE_EHIP, "%s: HIP error %d (%s)", where, (int)e, hipGetErrorString(e));
}

#define MOE_TRY(expr)                      \
  do {                                     \
    moe_status _s = (expr);                \
    if (_s != MOE_OK) return _s;           \
  } while (0)
#define MOE_HIP(expr, where) MOE_TRY(hip_status((expr), (where)))

// ---- stage timing (moe_timing_enable / moe_timing_read) ----
constexpr int kTimingSlots = 4096;
struct Timing {
  bool on = false;
  int used = 0;
  int stage[kTimingSlots];
  hipEvent_t ev0[kTimingSlots];
  hipEvent_t ev1[kTimingSlots];
  bool created = false;
};
Timing g_timing;

// Record the start of a stage: the slot, or -1 when timing is off or the slots are used up.
hipError_t stage_begin(int stage, hipStream_t st, int* slot) {
  *slot = -1;
  if (!g_timing.on || g_timing.used >= kTimingSlots) return hipSuccess;
  const int i = g_timing.used;
  const hipError_t e = hipEventRecord(g_timing.ev0[i], st);
  if (e != hipSuccess) return e;
  g_timing.stage[i] = stage;
  g_timing.used = i + 1;
  *slot = i;
  return hipSuccess;
}
hipError_t stage_end(int slot, hipStream_t st) {
  return slot >= 0 ? hipEventRecord(g_timing.ev1[slot], st) : hipSuccess;
}

// Run one stage's launcher between timing events; a failed launch or event record is MOE_EHIP.
#define MOE_STAGE(stage, st, expr, where)                      \
  do {                                                         \
    int _slot;                                                 \
    MOE_HIP(stage_begin((stage), (st), &_slot), "timing event"); \
    const hipError_t _e = (expr);                              \
    MOE_HIP(_e, where);                                        \
    MOE_HIP(stage_end(_slot, (st)), "timing event");           \
  } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moe_status need_ptr(const void* p, const char* name) {
  if (!p) return fail(MOE_EINVAL, "%s is NULL", name);
  if (!aligned16(p)) return fail(MOE_EINVAL, "%s is not 16-byte aligned", name);
  return MOE_OK;
}
moe_status opt_ptr(const void* p, const char* name) {
  if (p && !aligned16(p)) return fail(MOE_EINVAL, "%s is not 16-byte aligned", name);
  return MOE_OK;
}

moe_status check_dims(const moe_dims* dm) {
  if (!dm) return fail(MOE_EINVAL, "dims is NULL");
  if (dm->T < 1 || dm->T > (1 << 24)) return fail(MOE_EINVAL, "T=%lld out of range [1, 2^24]", (long long)dm->T);
  if (dm->E < 1 || dm->E > 1024) return fail(MOE_EINVAL, "E=%d out of range [1, 1024]", dm->E);
  if (dm->K < 1 || dm->K > dm->E) return fail(MOE_EINVAL, "K=%d out of range [1, E=%d]", dm->K, dm->E);
  if (dm->K > 16) return fail(MOE_ENOTSUP, "K=%d > 16 is not supported", dm->K);
  if (dm->d < 64 || dm->d > 65536 || dm->n < 64 || dm->n > 65536)
    return fail(MOE_EINVAL, "d=%lld / n=%lld out of range [64, 65536]", (long long)dm->d, (long long)dm->n);
  if (dm->d % 64 || dm->n % 64)
    return fail(MOE_ENOTSUP, "d=%lld and n=%lld must be multiples of 64", (long long)dm->d, (long long)dm->n);
  if (dm->dtype != MOE_F32 && dm->dtype != MOE_BF16) return fail(MOE_ENOTSUP, "dtype %d not supported", dm->dtype);
  if (dm->round_mode < MOE_ROUND_NONE || dm->round_mode > MOE_ROUND_STOCHASTIC)
    return fail(MOE_EINVAL, "round_mode %d invalid", dm->round_mode);
  if (dm->round_mode == MOE_ROUND_STOCHASTIC && !dm->round_rand)
    return fail(MOE_EINVAL, "MOE_ROUND_STOCHASTIC needs round_rand");
  if (dm->round_mode != MOE_ROUND_NONE && (dm->tile_m < 1 || dm->tile_m > 1024))
    return fail(MOE_EINVAL, "tile_m=%d out of range [1, 1024]", dm->tile_m);
  if (dm->flags != 0) return fail(MOE_EINVAL, "flags must be 0");
  return MOE_OK;
}

int64_t max_rows(const moe_dims* dm) {
  const int64_t base = dm->T * dm->K;
  if (dm->round_mode == MOE_ROUND_NONE || dm->round_mode == MOE_ROUND_DOWN) return base;
  const int64_t up = base + (int64_t)dm->E * (dm->tile_m - 1);
  const int64_t cap = dm->T * dm->E;
  return up < cap ? up : cap;
}

Shape shape_of(const moe_dims* dm) {
  Shape s;
  s.T = dm->T;
  s.d = dm->d;
  s.n = dm->n;
  s.E = dm->E;
  s.K = dm->K;
  s.R_max = max_rows(dm);
  s.bf16 = dm->dtype == MOE_BF16;
  return s;
}

size_t esize(const moe_dims* dm) { return dm->dtype == MOE_BF16 ? 2 : 4; }
int e_pad(int E) { return (E + 7) / 8 * 8; }

// Bump allocator over the workspace; with base == nullptr it only measures.
struct Carve {
  char* base;
  size_t off = 0;
  explicit Carve(void* b) : base(static_cast<char*>(b)) {}
  void* take(size_t bytes) {
    void* p = base ? base + off : nullptr;
    off = align_up(off + bytes, 256);
    return p;
  }
};

struct FfnWs {
  int32_t* mtile_off;
  void* act;
};
FfnWs carve_ffn(Carve& c, const moe_dims* dm) {
  FfnWs w;
  w.mtile_off = static_cast<int32_t*>(c.take((size_t)tile_table_ints(dm->E) * 4));
  w.act = c.take((size_t)max_rows(dm) * dm->n * esize(dm));
  return w;
}

struct BwdWs {
  int32_t* mtile_off;
  int32_t* order;
  void* H;
  void* dH;
  void* wA;
  float* dS_part;
  void* dX_perm;
  void* dLop;
  void* dwr;
};
BwdWs carve_bwd(Carve& c, const moe_dims* dm) {
  const Shape s = shape_of(dm);
  const size_t es = esize(dm);
  BwdWs w;
  w.mtile_off = static_cast<int32_t*>(c.take((size_t)tile_table_ints(dm->E) * 4));
  w.order = static_cast<int32_t*>(c.take((size_t)dm->E * 4));
  w.H = c.take((size_t)s.R_max * 2 * dm->n * es);
  w.dH = c.take((size_t)s.R_max * 2 * dm->n * es);
  w.wA = c.take((size_t)s.R_max * dm->n * es);
  w.dS_part = static_cast<float*>(c.take((size_t)dact_ntiles(dm->n) * s.R_max * 4));
  w.dX_perm = c.take((size_t)s.R_max * dm->d * es);
  w.dLop = c.take((size_t)dm->T * e_pad(dm->E) * es);
  w.dwr = c.take(dwr_workspace_bytes(s));
  return w;
}

size_t ws_bytes_for(const moe_dims* dm, int op) {
  Carve c(nullptr);
  switch (op) {
    case MOE_OP_ROUTE:  // (+ the partial products of a split router GEMM)
      return route_workspace_bytes(dm->T, dm->E, dm->round_mode != 0) + router_part_bytes(shape_of(dm));
    case MOE_OP_PERMUTE: return 0;
    case MOE_OP_COMBINE: return 0;
    case MOE_OP_FFN: carve_ffn(c, dm); return c.off;
    case MOE_OP_FORWARD: {
      carve_ffn(c, dm);
      c.take((size_t)max_rows(dm) * dm->d * esize(dm));  // Y_perm
      const size_t r = route_workspace_bytes(dm->T, dm->E, dm->round_mode != 0) + router_part_bytes(shape_of(dm));
      return c.off > r ? c.off : r;
    }
    case MOE_OP_BACKWARD: carve_bwd(c, dm); return c.off;
    case MOE_OP_DECODE: return decode_workspace_bytes(dm->T, dm->d, dm->n, dm->E, dm->K);
    case MOE_OP_FFN_FP8: c.take((size_t)tile_table_ints(dm->E) * 4); return c.off;
    case MOE_OP_FFN_MX:  // tile table, the token scales in routed-row order
      c.take((size_t)tile_table_ints(dm->E) * 4);
      c.take((size_t)mx_scale_bytes(max_rows(dm), dm->d));
      return c.off;
    default: return 0;
  }
}

moe_status check_plan(const moe_plan* p) {
  if (!p) return fail(MOE_EINVAL, "plan is NULL");
  MOE_TRY(need_ptr(p->topk_idx, "plan.topk_idx"));
  MOE_TRY(need_ptr(p->topk_w, "plan.topk_w"));
  MOE_TRY(need_ptr(p->counts, "plan.counts"));
  MOE_TRY(need_ptr(p->expert_off, "plan.expert_off"));
  MOE_TRY(need_ptr(p->row_token, "plan.row_token"));
  MOE_TRY(need_ptr(p->row_w, "plan.row_w"));
  MOE_TRY(need_ptr(p->tok_off, "plan.tok_off"));
  MOE_TRY(need_ptr(p->tok_row, "plan.tok_row"));
  MOE_TRY(need_ptr(p->meta, "plan.meta"));
  return MOE_OK;
}

PlanPtrs plan_ptrs(const moe_plan* p) {
  PlanPtrs q;
  q.topk_idx = p->topk_idx;
  q.topk_w = p->topk_w;
  q.counts = p->counts;
  q.expert_off = p->expert_off;
  q.row_token = p->row_token;
  q.row_w = p->row_w;
  q.tok_off = p->tok_off;
  q.tok_row = p->tok_row;
  q.meta = p->meta;
  return q;
}

moe_status check_ws(const moe_dims* dm, int op, void* ws, size_t ws_bytes) {
  const size_t need = ws_bytes_for(dm, op);
  if (need == 0) return MOE_OK;
  if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  return need_ptr(ws, "ws");
}

// The routing stage shared by moe_route and moe_forward (arguments already validated).
// With X the router GEMM runs first; when it splits its reduction (router_split), the partial
// products go to the end of the routing workspace and top-K adds them into logits.
moe_status do_route(const moe_dims* dm, const void* X, const void* W_r, const float* bias,
                    float* logits, const moe_plan* plan, void* ws, hipStream_t st) {
  const Shape s = shape_of(dm);
  const int SK = X ? router_split(s) : 1;
  float* part = SK > 1 ? reinterpret_cast<float*>(static_cast<char*>(ws) +
                                                  route_workspace_bytes(dm->T, dm->E, dm->round_mode != 0))
                       : nullptr;
  if (X) MOE_STAGE(MOE_STAGE_ROUTER_GEMM, st, launch_router_gemm(s, X, W_r, bias, logits, part, st), "router GEMM");
  MOE_STAGE(MOE_STAGE_ROUTE, st,
            launch_route(logits, part, SK, dm->T, dm->E, dm->K, dm->round_mode, dm->tile_m, dm->round_rand,
                         plan_ptrs(plan), ws, st),
            "routing");
  return MOE_OK;
}

moe_status do_ffn(const moe_dims* dm, const moe_plan* plan, const void* A_in, bool gathered,
                  const void* Wg, const void* Wu, const void* Wd, void* H, void* Y, const FfnWs& w,
                  hipStream_t st) {
  const Shape s = shape_of(dm);
  const PlanPtrs p = plan_ptrs(plan);
  MOE_STAGE(MOE_STAGE_TILES, st, launch_tile_offsets(p.counts, dm->E, w.mtile_off, nullptr, st), "tile offsets");
  MOE_STAGE(MOE_STAGE_UP_GEMM, st, launch_up_gemm(s, p, w.mtile_off, A_in, gathered, Wg, Wu, w.act, H, st),
            "gate/up GEMM");
  MOE_STAGE(MOE_STAGE_DOWN_GEMM, st, launch_down_gemm(s, p, w.mtile_off, w.act, Wd, Y, st), "down GEMM");
  return MOE_OK;
}

// ---- allocation-free routing (moe_route_noalloc) ----
// The routing workspace of moe_route_noalloc: one copy per device, held until the process ends.
// In host code `scratch` names a host-side stand-in, not device memory; kernels get the device
// address from hipGetSymbolAddress, resolved once per device.
constexpr size_t kRouteScratchBytes = size_t(64) << 20;
static __device__ __align__(256) char scratch[kRouteScratchBytes];

constexpr int kMaxDevices = 64;
void* g_scratch_ptr[kMaxDevices];
std::mutex g_scratch_mu;

moe_status route_scratch(void** out) {
  int dev = 0;
  MOE_HIP(hipGetDevice(&dev), "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(MOE_EHIP, "device %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    MOE_HIP(hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)), "hipGetSymbolAddress(scratch)");
    if (!p) return fail(MOE_EHIP, "hipGetSymbolAddress(scratch) returned NULL");
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_max_rows(const moe_dims* dims) {
  if (check_dims(dims) != MOE_OK) return 0;
  return max_rows(dims);
}

size_t moe_workspace_bytes(const moe_dims* dims, int op) {
  if (check_dims(dims) != MOE_OK) return 0;
  if (op < MOE_OP_ROUTE || op > MOE_OP_FFN_MX) {
    fail(MOE_EINVAL, "unknown op %d", op);
    return 0;
  }
  return ws_bytes_for(dims, op);
}

moe_status moe_route(const moe_dims* dims, const void* X, const void* W_r, const float* bias,
                     float* logits, const moe_plan* plan, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(logits, "logits"));
  if (X) {
    MOE_TRY(need_ptr(X, "X"));
    MOE_TRY(need_ptr(W_r, "W_r"));
    MOE_TRY(opt_ptr(bias, "bias"));
  }
  MOE_TRY(check_ws(dims, MOE_OP_ROUTE, ws, ws_bytes));
  return do_route(dims, X, W_r, bias, logits, plan, ws, static_cast<hipStream_t>(stream));
}

size_t moe_route_noalloc_max_bytes(void) { return kRouteScratchBytes; }

moe_status moe_route_noalloc(const moe_dims* dims, const void* X, const void* W_r, const float* bias,
                             float* logits, const moe_plan* plan, void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(logits, "logits"));
  if (X) {
    MOE_TRY(need_ptr(X, "X"));
    MOE_TRY(need_ptr(W_r, "W_r"));
    MOE_TRY(opt_ptr(bias, "bias"));
  }
  const size_t need = ws_bytes_for(dims, MOE_OP_ROUTE);
  if (need > kRouteScratchBytes)
    return fail(MOE_EWORKSPACE, "routing needs %zu bytes of workspace, more than the %zu of the static buffer",
                need, kRouteScratchBytes);
  void* ws = nullptr;
  MOE_TRY(route_scratch(&ws));
  return do_route(dims, X, W_r, bias, logits, plan, ws, static_cast<hipStream_t>(stream));
}

moe_status moe_permute(const moe_dims* dims, const moe_plan* plan, const void* X, void* X_perm,
                       void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(X, "X"));
  MOE_TRY(need_ptr(X_perm, "X_perm"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_PERMUTE, st, launch_permute(shape_of(dims), plan_ptrs(plan), X, X_perm, st), "permute");
  return MOE_OK;
}

moe_status moe_grouped_ffn(const moe_dims* dims, const moe_plan* plan, const void* A_in,
                           int gathered, const void* W_gate, const void* W_up,
                           const void* W_down, void* H_cache, void* Y_perm, void* ws,
                           size_t ws_bytes, void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(A_in, gathered ? "X" : "X_perm"));
  MOE_TRY(need_ptr(W_gate, "W_gate"));
  MOE_TRY(need_ptr(W_up, "W_up"));
  MOE_TRY(need_ptr(W_down, "W_down"));
  MOE_TRY(opt_ptr(H_cache, "H_cache"));
  MOE_TRY(need_ptr(Y_perm, "Y_perm"));
  MOE_TRY(check_ws(dims, MOE_OP_FFN, ws, ws_bytes));
  Carve c(ws);
  const FfnWs w = carve_ffn(c, dims);
  return do_ffn(dims, plan, A_in, gathered != 0, W_gate, W_up, W_down, H_cache, Y_perm, w,
                static_cast<hipStream_t>(stream));
}

moe_status moe_combine(const moe_dims* dims, const moe_plan* plan, const void* Y_perm,
                       int weighted, void* out, void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(Y_perm, "Y_perm"));
  MOE_TRY(need_ptr(out, "out"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_COMBINE, st, launch_combine(shape_of(dims), plan_ptrs(plan), Y_perm, weighted != 0, out, st),
            "combine");
  return MOE_OK;
}

moe_status moe_quantize_fp8(int64_t rows, int64_t K, int dtype, const void* src, uint8_t* codes,
                            float* scales, void* stream) {
  if (rows < 0 || rows > ((int64_t)1 << 31)) return fail(MOE_EINVAL, "rows=%lld out of range", (long long)rows);
  if (K < 8 || K > 65536 || K % 8) return fail(MOE_EINVAL, "K=%lld must be a multiple of 8 in [8, 65536]", (long long)K);
  if (dtype != MOE_BF16 && dtype != MOE_F32) return fail(MOE_ENOTSUP, "dtype %d not supported", dtype);
  if (rows == 0) return MOE_OK;
  MOE_TRY(need_ptr(src, "src"));
  MOE_TRY(need_ptr(codes, "codes"));
  MOE_TRY(need_ptr(scales, "scales"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_FP8_QUANT, st, launch_quant_fp8(src, dtype == MOE_BF16, rows, K, nullptr, codes, scales, st),
            "fp8 quantisation");
  return MOE_OK;
}

moe_status moe_grouped_ffn_fp8(const moe_dims* dims, const moe_plan* plan, const uint8_t* Xq,
                               const float* sx, const uint8_t* Wg_q, const float* sg,
                               const uint8_t* Wu_q, const float* su, const uint8_t* Wd_q,
                               const float* sd, void* act, uint8_t* act_q, float* sact,
                               void* Y_perm, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_dims(dims));
  if (dims->dtype != MOE_BF16) return fail(MOE_ENOTSUP, "moe_grouped_ffn_fp8 needs dtype MOE_BF16");
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(Xq, "Xq"));
  MOE_TRY(need_ptr(sx, "sx"));
  MOE_TRY(need_ptr(Wg_q, "Wg_q"));
  MOE_TRY(need_ptr(sg, "sg"));
  MOE_TRY(need_ptr(Wu_q, "Wu_q"));
  MOE_TRY(need_ptr(su, "su"));
  MOE_TRY(need_ptr(Wd_q, "Wd_q"));
  MOE_TRY(need_ptr(sd, "sd"));
  MOE_TRY(need_ptr(act, "act"));
  MOE_TRY(need_ptr(act_q, "act_q"));
  MOE_TRY(need_ptr(sact, "sact"));
  MOE_TRY(need_ptr(Y_perm, "Y_perm"));
  MOE_TRY(check_ws(dims, MOE_OP_FFN_FP8, ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Shape s = shape_of(dims);
  const PlanPtrs p = plan_ptrs(plan);
  int32_t* mtile_off = static_cast<int32_t*>(ws);
  MOE_STAGE(MOE_STAGE_TILES, st, launch_tile_offsets(p.counts, dims->E, mtile_off, nullptr, st), "tile offsets");
  MOE_STAGE(MOE_STAGE_FP8_UP, st, launch_up_fp8(s, p, mtile_off, Xq, sx, Wg_q, sg, Wu_q, su, act, st),
            "fp8 gate/up GEMM");
  MOE_STAGE(MOE_STAGE_FP8_QUANT, st, launch_quant_fp8(act, true, s.R_max, dims->n, p.meta, act_q, sact, st),
            "fp8 activation quantisation");
  MOE_STAGE(MOE_STAGE_FP8_DOWN, st, launch_down_fp8(s, p, mtile_off, act_q, sact, Wd_q, sd, Y_perm, st),
            "fp8 down GEMM");
  return MOE_OK;
}

moe_status moe_decode(const moe_dims* dims, const void* X, const void* W_r, const float* bias,
                      const void* W_gate, const void* W_up, const void* W_down, float* logits,
                      int32_t* topk_idx, float* topk_w, void* out, void* ws, size_t ws_bytes,
                      void* stream) {
  MOE_TRY(check_dims(dims));
  if (dims->round_mode != MOE_ROUND_NONE)
    return fail(MOE_ENOTSUP, "moe_decode routes with plain top-K (round_mode must be NONE)");
  if (dims->T > 1024) return fail(MOE_ENOTSUP, "moe_decode handles T <= 1024 (got %lld)", (long long)dims->T);
  MOE_TRY(need_ptr(X, "X"));
  MOE_TRY(need_ptr(W_r, "W_r"));
  MOE_TRY(opt_ptr(bias, "bias"));
  MOE_TRY(need_ptr(W_gate, "W_gate"));
  MOE_TRY(need_ptr(W_up, "W_up"));
  MOE_TRY(need_ptr(W_down, "W_down"));
  MOE_TRY(need_ptr(logits, "logits"));
  MOE_TRY(need_ptr(topk_idx, "topk_idx"));
  MOE_TRY(need_ptr(topk_w, "topk_w"));
  MOE_TRY(need_ptr(out, "out"));
  MOE_TRY(check_ws(dims, MOE_OP_DECODE, ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_DECODE, st,
            launch_decode(shape_of(dims), X, W_r, bias, W_gate, W_up, W_down, logits, topk_idx,
                          topk_w, out, ws, st),
            "decode");
  return MOE_OK;
}

int64_t moe_mx_scale_bytes(int64_t rows, int64_t K) { return rows >= 0 && K > 0 ? mx_scale_bytes(rows, K) : 0; }

moe_status moe_quantize_mx(int64_t rows, int64_t K, int dtype, int fmt, const void* src, uint8_t* codes,
                           uint8_t* scales, void* stream) {
  if (rows < 0 || rows > ((int64_t)1 << 31)) return fail(MOE_EINVAL, "rows=%lld out of range", (long long)rows);
  if (K < 64 || K > 65536 || K % 64) return fail(MOE_EINVAL, "K=%lld must be a multiple of 64 in [64, 65536]", (long long)K);
  if (dtype != MOE_BF16 && dtype != MOE_F32) return fail(MOE_ENOTSUP, "dtype %d not supported", dtype);
  if (fmt != MOE_FP8_E4M3 && fmt != MOE_FP8_E5M2) return fail(MOE_EINVAL, "fp8 format %d invalid", fmt);
  if (rows == 0) return MOE_OK;
  MOE_TRY(need_ptr(src, "src"));
  MOE_TRY(need_ptr(codes, "codes"));
  MOE_TRY(need_ptr(scales, "scales"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_FP8_QUANT, st, launch_quant_mx(src, dtype == MOE_BF16, fmt, rows, K, codes, scales, st),
            "block-scaled fp8 quantisation");
  return MOE_OK;
}

moe_status moe_grouped_ffn_mx(const moe_dims* dims, const moe_plan* plan, int fmt, const uint8_t* Xq,
                              const uint8_t* sx, const uint8_t* Wg_q, const uint8_t* sg, const uint8_t* Wu_q,
                              const uint8_t* su, const uint8_t* Wd_q, const uint8_t* sd, void* act,
                              uint8_t* act_q, uint8_t* sact, void* Y_perm, void* ws, size_t ws_bytes,
                              void* stream) {
  MOE_TRY(check_dims(dims));
  if (dims->dtype != MOE_BF16) return fail(MOE_ENOTSUP, "moe_grouped_ffn_mx needs dtype MOE_BF16");
  if (fmt != MOE_FP8_E4M3 && fmt != MOE_FP8_E5M2) return fail(MOE_EINVAL, "fp8 format %d invalid", fmt);
  if (dims->T * dims->d >= ((int64_t)1 << 32))
    return fail(MOE_ENOTSUP, "moe_grouped_ffn_mx needs T * d < 2^32 (T=%lld, d=%lld)", (long long)dims->T,
                (long long)dims->d);
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(Xq, "Xq"));
  MOE_TRY(need_ptr(sx, "sx"));
  MOE_TRY(need_ptr(Wg_q, "Wg_q"));
  MOE_TRY(need_ptr(sg, "sg"));
  MOE_TRY(need_ptr(Wu_q, "Wu_q"));
  MOE_TRY(need_ptr(su, "su"));
  MOE_TRY(need_ptr(Wd_q, "Wd_q"));
  MOE_TRY(need_ptr(sd, "sd"));
  MOE_TRY(opt_ptr(act, "act"));
  MOE_TRY(need_ptr(act_q, "act_q"));
  MOE_TRY(need_ptr(sact, "sact"));
  MOE_TRY(need_ptr(Y_perm, "Y_perm"));
  MOE_TRY(check_ws(dims, MOE_OP_FFN_MX, ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Shape s = shape_of(dims);
  const PlanPtrs p = plan_ptrs(plan);
  Carve c(ws);
  int32_t* mtile_off = static_cast<int32_t*>(c.take((size_t)tile_table_ints(dims->E) * 4));
  uint8_t* sxp = static_cast<uint8_t*>(c.take((size_t)mx_scale_bytes(s.R_max, dims->d)));
  MOE_STAGE(MOE_STAGE_TILES, st, launch_tile_offsets(p.counts, dims->E, mtile_off, nullptr, st), "tile offsets");
  MOE_STAGE(MOE_STAGE_FP8_QUANT, st, launch_gather_mx_scales(s, p, sx, sxp, st), "token scale gather");
  MOE_STAGE(MOE_STAGE_FP8_UP, st,
            launch_up_mx(s, p, mtile_off, fmt, Xq, sxp, Wg_q, sg, Wu_q, su, act, act_q, sact, st),
            "block-scaled fp8 gate/up GEMM");
  MOE_STAGE(MOE_STAGE_FP8_DOWN, st, launch_down_mx(s, p, mtile_off, fmt, act_q, sact, Wd_q, sd, Y_perm, st),
            "block-scaled fp8 down GEMM");
  return MOE_OK;
}

moe_status moe_decode_status(void* stream) {
  int failed = 0;
  MOE_HIP(decode_read_status(static_cast<hipStream_t>(stream), &failed), "moe_decode_status");
  if (failed)
    return fail(MOE_EHIP, "moe_decode: a workgroup gave up waiting at a grid barrier; the outputs of "
                          "that call are invalid");
  return MOE_OK;
}

long long moe_decode_set_spin_limit(long long limit) {
  if (limit < 0) {
    fail(MOE_EINVAL, "spin limit %lld < 0", limit);
    return -1;
  }
  return decode_set_spin_limit(limit);
}

moe_status moe_forward(const moe_dims* dims, const void* X, const void* W_r, const float* bias,
                       const void* W_gate, const void* W_up, const void* W_down, float* logits,
                       const moe_plan* plan, void* H_cache, void* out, void* ws, size_t ws_bytes,
                       void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(X, "X"));
  MOE_TRY(need_ptr(W_r, "W_r"));
  MOE_TRY(opt_ptr(bias, "bias"));
  MOE_TRY(need_ptr(W_gate, "W_gate"));
  MOE_TRY(need_ptr(W_up, "W_up"));
  MOE_TRY(need_ptr(W_down, "W_down"));
  MOE_TRY(need_ptr(logits, "logits"));
  MOE_TRY(opt_ptr(H_cache, "H_cache"));
  MOE_TRY(need_ptr(out, "out"));
  MOE_TRY(check_ws(dims, MOE_OP_FORWARD, ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_TRY(do_route(dims, X, W_r, bias, logits, plan, ws, st));
  Carve c(ws);
  const FfnWs w = carve_ffn(c, dims);
  void* Y = c.take((size_t)max_rows(dims) * dims->d * esize(dims));
  MOE_TRY(do_ffn(dims, plan, X, true, W_gate, W_up, W_down, H_cache, Y, w, st));
  MOE_STAGE(MOE_STAGE_COMBINE, st, launch_combine(shape_of(dims), plan_ptrs(plan), Y, true, out, st), "combine");
  return MOE_OK;
}

moe_status moe_backward(const moe_dims* dims, const void* dY, const void* X, const void* W_r,
                        const void* W_gate, const void* W_up, const void* W_down,
                        const moe_plan* plan, const void* H_cache, void* dX, void* dW_gate,
                        void* dW_up, void* dW_down, float* dS, float* dLogits, void* dW_r,
                        void* ws, size_t ws_bytes, void* stream) {
  return moe_backward_aux(dims, dY, X, W_r, W_gate, W_up, W_down, plan, H_cache, nullptr, dX, dW_gate, dW_up, dW_down,
                          dS, dLogits, dW_r, ws, ws_bytes, stream);
}

moe_status moe_backward_aux(const moe_dims* dims, const void* dY, const void* X, const void* W_r,
                            const void* W_gate, const void* W_up, const void* W_down,
                            const moe_plan* plan, const void* H_cache, const float* dLogits_aux, void* dX,
                            void* dW_gate, void* dW_up, void* dW_down, float* dS, float* dLogits, void* dW_r,
                            void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(dY, "dY"));
  MOE_TRY(need_ptr(X, "X"));
  MOE_TRY(opt_ptr(W_r, "W_r"));
  MOE_TRY(need_ptr(W_gate, "W_gate"));
  MOE_TRY(need_ptr(W_up, "W_up"));
  MOE_TRY(need_ptr(W_down, "W_down"));
  MOE_TRY(opt_ptr(H_cache, "H_cache"));
  MOE_TRY(opt_ptr(dLogits_aux, "dLogits_aux"));
  if (dLogits_aux && dLogits_aux == dLogits) return fail(MOE_EINVAL, "dLogits_aux must not be the dLogits array");
  MOE_TRY(need_ptr(dX, "dX"));
  MOE_TRY(need_ptr(dW_gate, "dW_gate"));
  MOE_TRY(need_ptr(dW_up, "dW_up"));
  MOE_TRY(need_ptr(dW_down, "dW_down"));
  MOE_TRY(need_ptr(dS, "dS"));
  MOE_TRY(need_ptr(dLogits, "dLogits"));
  MOE_TRY(opt_ptr(dW_r, "dW_r"));
  if (dW_r && !W_r) return fail(MOE_EINVAL, "dW_r requested without W_r");
  MOE_TRY(check_ws(dims, MOE_OP_BACKWARD, ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Shape s = shape_of(dims);
  const PlanPtrs p = plan_ptrs(plan);
  Carve c(ws);
  const BwdWs w = carve_bwd(c, dims);
  MOE_STAGE(MOE_STAGE_TILES, st, launch_tile_offsets(p.counts, dims->E, w.mtile_off, w.order, st),
            "tile offsets and expert order");
  const void* H = H_cache;
  if (!H) {  // recompute [G | U] from X; the SwiGLU output goes to wA, which dAct overwrites
    MOE_STAGE(MOE_STAGE_UP_GEMM, st, launch_up_gemm(s, p, w.mtile_off, X, true, W_gate, W_up, w.wA, w.H, st),
              "recompute GEMM");
    H = w.H;
  }
  MOE_STAGE(MOE_STAGE_DACT_GEMM, st,
            launch_dact_gemm(s, p, w.mtile_off, dY, W_down, H, w.dH, w.wA, w.dS_part, st), "dAct GEMM");
  MOE_STAGE(MOE_STAGE_DW_DOWN_GEMM, st, launch_dw_down_gemm(s, p, w.order, dY, w.wA, dW_down, st), "dW_down GEMM");
  MOE_STAGE(MOE_STAGE_DW_GU_GEMM, st, launch_dw_gu_gemm(s, p, w.order, w.dH, X, dW_gate, dW_up, st),
            "dW_gate/up GEMM");
  MOE_STAGE(MOE_STAGE_DX_GEMM, st, launch_dx_gemm(s, p, w.mtile_off, w.dH, W_gate, W_up, w.dX_perm, st),
            "dX GEMM");
  MOE_STAGE(MOE_STAGE_ROUTER_BWD, st,
            launch_router_bwd(s, p, w.dS_part, dact_ntiles(dims->n), w.dX_perm, dLogits_aux ? nullptr : W_r,
                              dLogits_aux, dS, dLogits, dW_r || (dLogits_aux && W_r) ? w.dLop : nullptr,
                              e_pad(dims->E), dX, st),
            "router backward");
  if (dLogits_aux && W_r)  // dense logit gradients: their dX term is a GEMM that adds to the gathered sum
    MOE_STAGE(MOE_STAGE_LINEAR_BWD, st, launch_logit_dx(s, w.dLop, e_pad(dims->E), W_r, dX, st), "logit dX GEMM");
  if (dW_r)
    MOE_STAGE(MOE_STAGE_DWR_GEMM, st, launch_dwr_gemm(s, w.dLop, e_pad(dims->E), X, dW_r, w.dwr, st),
              "dW_r GEMM");
  return MOE_OK;
}

// ---- router losses ----
static moe_status check_n_seq(int32_t n_seq) {
  if (n_seq < 1 || n_seq > (1 << 20)) return fail(MOE_EINVAL, "n_seq=%d out of range [1, 2^20]", n_seq);
  return MOE_OK;
}
static moe_status check_sequences(int32_t n_seq, const int32_t* seq_off, const uint8_t* mask) {
  MOE_TRY(check_n_seq(n_seq));
  if (n_seq > 1 && !seq_off) return fail(MOE_EINVAL, "n_seq=%d needs seq_off", n_seq);
  MOE_TRY(opt_ptr(seq_off, "seq_off"));
  return opt_ptr(mask, "token_mask");
}

size_t moe_router_loss_workspace_bytes(const moe_dims* dims, int32_t n_seq) {
  if (check_dims(dims) != MOE_OK || check_n_seq(n_seq) != MOE_OK) return 0;
  return router_loss_workspace_bytes(dims->T, dims->E, n_seq);
}

moe_status moe_router_loss(const moe_dims* dims, const float* logits, const int32_t* topk_idx, int32_t n_seq,
                           const int32_t* seq_off, const uint8_t* token_mask, int32_t* seq_tokens,
                           int32_t* seq_counts, float* prob_sum, float* lse, float* loss, void* ws, size_t ws_bytes,
                           void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_sequences(n_seq, seq_off, token_mask));
  MOE_TRY(need_ptr(logits, "logits"));
  MOE_TRY(need_ptr(topk_idx, "topk_idx"));
  MOE_TRY(need_ptr(seq_tokens, "seq_tokens"));
  MOE_TRY(need_ptr(seq_counts, "seq_counts"));
  MOE_TRY(need_ptr(prob_sum, "prob_sum"));
  MOE_TRY(need_ptr(lse, "lse"));
  MOE_TRY(need_ptr(loss, "loss"));
  const size_t need = router_loss_workspace_bytes(dims->T, dims->E, n_seq);
  if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  MOE_TRY(need_ptr(ws, "ws"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_ROUTER_LOSS, st,
            launch_router_loss(logits, topk_idx, dims->T, dims->E, dims->K, n_seq, seq_off, token_mask, seq_tokens,
                               seq_counts, prob_sum, lse, loss, ws, st),
            "router loss");
  return MOE_OK;
}

moe_status moe_router_loss_backward(const moe_dims* dims, const float* dloss, const float* logits, int32_t n_seq,
                                    const int32_t* seq_off, const uint8_t* token_mask, const int32_t* seq_tokens,
                                    const int32_t* seq_counts, const float* lse, float* dLogits, void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_sequences(n_seq, seq_off, token_mask));
  MOE_TRY(need_ptr(dloss, "dloss"));
  MOE_TRY(need_ptr(logits, "logits"));
  MOE_TRY(need_ptr(seq_tokens, "seq_tokens"));
  MOE_TRY(need_ptr(seq_counts, "seq_counts"));
  MOE_TRY(need_ptr(lse, "lse"));
  MOE_TRY(need_ptr(dLogits, "dLogits"));
  if (dLogits == logits) return fail(MOE_EINVAL, "dLogits must not be the logits array");
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_ROUTER_LOSS, st,
            launch_router_loss_bwd(dloss, logits, dims->T, dims->E, dims->K, n_seq, seq_off, token_mask, seq_tokens,
                                   seq_counts, lse, dLogits, st),
            "router loss backward");
  return MOE_OK;
}

// ---- dropout ----
static moe_status drop_args(double p, const uint64_t* rng, DropArgs* a) {
  if (!(p >= 0.0 && p <= 1.0)) return fail(MOE_EINVAL, "dropout probability %g out of range [0, 1]", p);
  MOE_TRY(need_ptr(rng, "rng"));
  a->rng = rng;
  a->threshold = static_cast<uint32_t>(p * 65536.0 + 0.5);
  a->scale = a->threshold < 65536u ? static_cast<float>(65536.0 / (65536.0 - a->threshold)) : 0.0f;
  return MOE_OK;
}

static moe_status check_ld(int64_t ld, int64_t cols, int64_t most, const char* name) {
  if (ld < cols || ld > most)
    return fail(MOE_EINVAL, "%s=%lld out of range [%lld, %lld]", name, (long long)ld, (long long)cols, (long long)most);
  return MOE_OK;
}
constexpr int64_t kMaxStride = (int64_t)1 << 40;        // dropout: 64-bit offsets throughout
constexpr int64_t kMaxLinearStride = (int64_t)1 << 22;  // dense projection: a tile's offsets are 32-bit

moe_status moe_dropout(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, const void* residual,
                       int64_t ldr, double p, const uint64_t* rng, void* out, int64_t ldo, void* stream) {
  if (rows < 0 || cols < 1 || cols > ((int64_t)1 << 30))
    return fail(MOE_EINVAL, "rows=%lld / cols=%lld out of range", (long long)rows, (long long)cols);
  if (rows > 0x7fffffffll || rows * ((cols + 7) / 8) > 0x7fffffffll)
    return fail(MOE_ENOTSUP, "rows=%lld x cols=%lld is more than 2^31 groups of 8", (long long)rows, (long long)cols);
  if (dtype != MOE_BF16 && dtype != MOE_F32) return fail(MOE_ENOTSUP, "dtype %d not supported", dtype);
  MOE_TRY(check_ld(ldx, cols, kMaxStride, "ldx"));
  MOE_TRY(check_ld(ldo, cols, kMaxStride, "ldo"));
  if (residual) MOE_TRY(check_ld(ldr, cols, kMaxStride, "ldr"));
  DropArgs a;
  MOE_TRY(drop_args(p, rng, &a));
  if (rows == 0) return MOE_OK;
  MOE_TRY(need_ptr(x, "x"));
  MOE_TRY(opt_ptr(residual, "residual"));
  MOE_TRY(need_ptr(out, "out"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_DROPOUT, st, launch_dropout(dtype == MOE_BF16, rows, cols, x, ldx, residual, ldr, out, ldo, a, st),
            "dropout");
  return MOE_OK;
}

moe_status moe_combine_dropout(const moe_dims* dims, const moe_plan* plan, const void* Y_perm, int weighted,
                               const void* residual, double p, const uint64_t* rng, void* out, void* stream) {
  MOE_TRY(check_dims(dims));
  MOE_TRY(check_plan(plan));
  MOE_TRY(need_ptr(Y_perm, "Y_perm"));
  MOE_TRY(opt_ptr(residual, "residual"));
  MOE_TRY(need_ptr(out, "out"));
  DropArgs a;
  MOE_TRY(drop_args(p, rng, &a));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_COMBINE, st,
            launch_combine_dropout(shape_of(dims), plan_ptrs(plan), Y_perm, weighted != 0, residual, out, a, st),
            "combine with dropout");
  return MOE_OK;
}

// ---- dense projection ----
static moe_status check_linear(const moe_linear_dims* dm, LinShape* s) {
  if (!dm) return fail(MOE_EINVAL, "dims is NULL");
  if (dm->M < 0 || dm->M > (1 << 24)) return fail(MOE_EINVAL, "M=%lld out of range [0, 2^24]", (long long)dm->M);
  if (dm->N < 8 || dm->N > 65536 || dm->K < 8 || dm->K > 65536)
    return fail(MOE_EINVAL, "N=%lld / K=%lld out of range [8, 65536]", (long long)dm->N, (long long)dm->K);
  if (dm->N % 8 || dm->K % 8)
    return fail(MOE_ENOTSUP, "N=%lld and K=%lld must be multiples of 8", (long long)dm->N, (long long)dm->K);
  if (dm->dtype != MOE_F32 && dm->dtype != MOE_BF16) return fail(MOE_ENOTSUP, "dtype %d not supported", dm->dtype);
  if (dm->act < MOE_ACT_NONE || dm->act > MOE_ACT_SWIGLU) return fail(MOE_EINVAL, "activation %d invalid", dm->act);
  if (dm->flags != 0) return fail(MOE_EINVAL, "flags must be 0");
  s->M = dm->M;
  s->N = dm->N;
  s->K = dm->K;
  s->ldx = dm->ldx ? dm->ldx : dm->K;
  s->ldr = dm->ldr ? dm->ldr : dm->N;
  s->ldy = dm->ldy ? dm->ldy : dm->N;
  s->act = dm->act;
  s->bf16 = dm->dtype == MOE_BF16;
  MOE_TRY(check_ld(s->ldx, s->K, kMaxLinearStride, "ldx"));
  MOE_TRY(check_ld(s->ldr, s->N, kMaxLinearStride, "ldr"));
  MOE_TRY(check_ld(s->ldy, s->N, kMaxLinearStride, "ldy"));
  if (s->ldx % 8 || s->ldr % 8 || s->ldy % 8)
    return fail(MOE_ENOTSUP, "ldx=%lld, ldr=%lld and ldy=%lld must be multiples of 8", (long long)s->ldx,
                (long long)s->ldr, (long long)s->ldy);
  return MOE_OK;
}

size_t moe_linear_workspace_bytes(const moe_linear_dims* dims, int op) {
  LinShape s;
  if (check_linear(dims, &s) != MOE_OK) return 0;
  if (op == MOE_LINEAR_FORWARD) return linear_fwd_workspace_bytes(s);
  if (op == MOE_LINEAR_BACKWARD) return linear_bwd_workspace_bytes(s);
  fail(MOE_EINVAL, "unknown op %d", op);
  return 0;
}

int moe_linear_plan(const moe_linear_dims* dims, int product, int32_t* slices, int32_t* paired) {
  LinShape s;
  MOE_TRY(check_linear(dims, &s));
  if (product < MOE_LINEAR_OUT || product > MOE_LINEAR_DW) return fail(MOE_EINVAL, "unknown product %d", product);
  int parts;
  bool both;
  const int tile = linear_plan(s, product, &parts, &both);
  if (slices) *slices = parts;
  if (paired) *paired = both ? 1 : 0;
  return tile;
}

static moe_status check_linear_ws(size_t need, void* ws, size_t ws_bytes) {
  if (need == 0) return MOE_OK;
  if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  return need_ptr(ws, "ws");
}

moe_status moe_linear(const moe_linear_dims* dims, const void* X, const void* W, const float* bias,
                      const void* residual, void* Z, void* out, void* ws, size_t ws_bytes, void* stream) {
  LinShape s;
  MOE_TRY(check_linear(dims, &s));
  if (s.M == 0) return MOE_OK;
  MOE_TRY(need_ptr(X, "X"));
  MOE_TRY(need_ptr(W, "W"));
  MOE_TRY(opt_ptr(bias, "bias"));
  MOE_TRY(opt_ptr(residual, "residual"));
  MOE_TRY(opt_ptr(Z, "Z"));
  MOE_TRY(need_ptr(out, "out"));
  MOE_TRY(check_linear_ws(linear_fwd_workspace_bytes(s), ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_LINEAR, st, launch_linear(s, X, W, bias, residual, Z, out, ws, st), "linear");
  return MOE_OK;
}

moe_status moe_linear_backward(const moe_linear_dims* dims, const void* dY, const void* X, const void* W,
                               const void* Z, void* dX, void* dW, float* dbias, void* ws, size_t ws_bytes,
                               void* stream) {
  LinShape s;
  MOE_TRY(check_linear(dims, &s));
  if (!dX && !dW && !dbias) return fail(MOE_EINVAL, "dX, dW and dbias are all NULL");
  if (s.M > 0) {
    MOE_TRY(need_ptr(dY, "dY"));
    if (dW) MOE_TRY(need_ptr(X, "X"));
    if (dX) MOE_TRY(need_ptr(W, "W"));
    if (s.act != MOE_ACT_NONE) MOE_TRY(need_ptr(Z, "Z"));
  }
  MOE_TRY(opt_ptr(dX, "dX"));
  MOE_TRY(opt_ptr(dW, "dW"));
  MOE_TRY(opt_ptr(dbias, "dbias"));
  MOE_TRY(check_linear_ws(linear_bwd_workspace_bytes(s), ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_LINEAR_BWD, st,
            launch_linear_bwd(s, dY, X, W, Z, s.M > 0 ? dX : nullptr, dW, dbias, ws, st), "linear backward");
  return MOE_OK;
}

// ---- layer / RMS norm ----
static moe_status check_norm(const moe_norm_dims* dm, NormShape* s) {
  if (!dm) return fail(MOE_EINVAL, "dims is NULL");
  if (dm->rows < 0 || dm->rows > 0x7fffffffll) return fail(MOE_EINVAL, "rows=%lld out of range [0, 2^31)", (long long)dm->rows);
  if (dm->cols < 1 || dm->cols > 65536) return fail(MOE_EINVAL, "cols=%lld out of range [1, 65536]", (long long)dm->cols);
  if (dm->dtype != MOE_F32 && dm->dtype != MOE_BF16) return fail(MOE_ENOTSUP, "dtype %d not supported", dm->dtype);
  if (dm->wtype != MOE_F32 && dm->wtype != MOE_BF16) return fail(MOE_ENOTSUP, "wtype %d not supported", dm->wtype);
  if (dm->kind != MOE_NORM_LAYER && dm->kind != MOE_NORM_RMS) return fail(MOE_EINVAL, "norm kind %d invalid", dm->kind);
  if (!(dm->eps >= 0.0f && dm->eps <= 3.4e38f)) return fail(MOE_EINVAL, "eps=%g must be finite and >= 0", (double)dm->eps);
  if (dm->flags != 0) return fail(MOE_EINVAL, "flags must be 0");
  s->rows = dm->rows;
  s->cols = dm->cols;
  s->ldx = dm->ldx ? dm->ldx : dm->cols;
  s->ldr = dm->ldr ? dm->ldr : dm->cols;
  s->lds = dm->lds ? dm->lds : dm->cols;
  s->ldy = dm->ldy ? dm->ldy : dm->cols;
  s->eps = dm->eps;
  s->bf16 = dm->dtype == MOE_BF16;
  s->wbf16 = dm->wtype == MOE_BF16;
  s->rms = dm->kind == MOE_NORM_RMS;
  MOE_TRY(check_ld(s->ldx, s->cols, kMaxStride, "ldx"));
  MOE_TRY(check_ld(s->ldr, s->cols, kMaxStride, "ldr"));
  MOE_TRY(check_ld(s->lds, s->cols, kMaxStride, "lds"));
  return check_ld(s->ldy, s->cols, kMaxStride, "ldy");
}
// An output that is an input's array takes its rows from the same places.
static moe_status check_alias(const void* out, int64_t ldo, const void* in, int64_t ldi, const char* name) {
  if (out && out == in && ldo != ldi) return fail(MOE_EINVAL, "%s is an input's array with another row stride", name);
  return MOE_OK;
}

moe_status moe_norm(const moe_norm_dims* dims, const void* x, const void* residual, const void* weight,
                    const void* bias, void* sum, void* y, float* mean, float* rstd, void* stream) {
  NormShape s;
  MOE_TRY(check_norm(dims, &s));
  if (s.rows == 0) return MOE_OK;
  MOE_TRY(need_ptr(x, "x"));
  MOE_TRY(opt_ptr(residual, "residual"));
  MOE_TRY(opt_ptr(weight, "weight"));
  MOE_TRY(opt_ptr(bias, "bias"));
  MOE_TRY(opt_ptr(sum, "sum"));
  MOE_TRY(need_ptr(y, "y"));
  MOE_TRY(opt_ptr(mean, "mean"));
  MOE_TRY(opt_ptr(rstd, "rstd"));
  if (sum && !residual) return fail(MOE_EINVAL, "sum requested without a residual");
  if (sum == y) return fail(MOE_EINVAL, "sum and y are the same array");
  MOE_TRY(check_alias(y, s.ldy, x, s.ldx, "y"));
  MOE_TRY(check_alias(y, s.ldy, residual, s.ldr, "y"));
  MOE_TRY(check_alias(sum, s.lds, x, s.ldx, "sum"));
  MOE_TRY(check_alias(sum, s.lds, residual, s.ldr, "sum"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_NORM, st, launch_norm(s, x, residual, weight, bias, sum, y, mean, rstd, st), "norm");
  return MOE_OK;
}

size_t moe_norm_workspace_bytes(const moe_norm_dims* dims) {
  NormShape s;
  return check_norm(dims, &s) == MOE_OK ? norm_bwd_workspace_bytes(s) : 0;
}

moe_status moe_norm_backward(const moe_norm_dims* dims, const void* dy, const void* sum, const void* weight,
                             const float* mean, const float* rstd, const void* dsum, void* dx, float* dweight,
                             float* dbias, void* ws, size_t ws_bytes, void* stream) {
  NormShape s;
  MOE_TRY(check_norm(dims, &s));
  if (!dx && !dweight && !dbias) return fail(MOE_EINVAL, "dx, dweight and dbias are all NULL");
  if (s.rows > 0) {
    MOE_TRY(need_ptr(dy, "dy"));
    MOE_TRY(need_ptr(sum, "s"));
    MOE_TRY(opt_ptr(weight, "weight"));
    if (!s.rms) MOE_TRY(need_ptr(mean, "mean"));
    MOE_TRY(need_ptr(rstd, "rstd"));
    MOE_TRY(opt_ptr(dsum, "dsum"));
  }
  MOE_TRY(opt_ptr(dx, "dx"));
  MOE_TRY(opt_ptr(dweight, "dweight"));
  MOE_TRY(opt_ptr(dbias, "dbias"));
  MOE_TRY(check_alias(dx, s.ldx, dy, s.ldy, "dx"));
  MOE_TRY(check_alias(dx, s.ldx, sum, s.lds, "dx"));
  MOE_TRY(check_alias(dx, s.ldx, dsum, s.ldr, "dx"));
  if (dweight && dweight == dbias) return fail(MOE_EINVAL, "dweight and dbias are the same array");
  if (dweight || dbias) {
    const size_t need = norm_bwd_workspace_bytes(s);
    if (need > 0) {
      if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
      MOE_TRY(need_ptr(ws, "ws"));
    }
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_NORM, st,
            launch_norm_bwd(s, dy, sum, weight, mean, rstd, dsum, dx, dweight, dbias, ws, st), "norm backward");
  return MOE_OK;
}

// ---- gradient norm and clipping ----
constexpr int32_t kMaxGrads = 1 << 16;
static moe_status check_grads(const moe_grad* g, int32_t count, GradTensor* out, int64_t* chunks) {
  *chunks = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].dtype != MOE_F32 && g[i].dtype != MOE_BF16) return fail(MOE_ENOTSUP, "tensor %d: dtype %d not supported", i, g[i].dtype);
    if (g[i].n < 0 || g[i].n > ((int64_t)1 << 36)) return fail(MOE_EINVAL, "tensor %d: n=%lld out of range [0, 2^36]", i, (long long)g[i].n);
    if (g[i].reserved != 0) return fail(MOE_EINVAL, "tensor %d: reserved must be 0", i);
    GradTensor t;
    t.src = g[i].src;
    t.dst = g[i].dst ? g[i].dst : const_cast<void*>(g[i].src);
    t.n = g[i].n;
    t.bf16 = g[i].dtype == MOE_BF16;
    const uintptr_t both = reinterpret_cast<uintptr_t>(t.src) | reinterpret_cast<uintptr_t>(t.dst);
    if (t.n > 0 && !t.src) return fail(MOE_EINVAL, "tensor %d: src is NULL", i);
    if (t.n > 0 && both % (t.bf16 ? 2 : 4)) return fail(MOE_EINVAL, "tensor %d is not aligned to its elements", i);
    *chunks += cdiv(t.n, GRAD_CHUNK);
    out[i] = t;
  }
  if (*chunks > 0x7fffffffll) return fail(MOE_ENOTSUP, "the tensors hold more than 2^31 chunks of %d elements", GRAD_CHUNK);
  return MOE_OK;
}
static size_t grad_table_bytes(int32_t count, int64_t chunks) { return (size_t)count * sizeof(GradEntry) + (size_t)chunks * 4; }
static moe_status grad_list(const moe_grad* g, int32_t count, std::unique_ptr<GradTensor[]>* out, int64_t* chunks) {
  if (count < 0 || count > kMaxGrads) return fail(MOE_EINVAL, "count=%d out of range [0, 2^16]", count);
  if (count > 0 && !g) return fail(MOE_EINVAL, "grads is NULL");
  out->reset(new (std::nothrow) GradTensor[count + 1]);
  if (!*out) return fail(MOE_EINVAL, "no host memory for %d tensors", count);
  return check_grads(g, count, out->get(), chunks);
}

size_t moe_grad_table_bytes(const moe_grad* grads, int32_t count) {
  std::unique_ptr<GradTensor[]> list;
  int64_t chunks = 0;
  if (grad_list(grads, count, &list, &chunks) != MOE_OK) return 0;
  const size_t bytes = grad_table_bytes(count, chunks);
  return bytes ? bytes : sizeof(GradEntry);
}

moe_status moe_grad_table(const moe_grad* grads, int32_t count, void* host_table, size_t bytes, moe_grad_list* out) {
  std::unique_ptr<GradTensor[]> list;
  int64_t chunks = 0;
  MOE_TRY(grad_list(grads, count, &list, &chunks));
  if (!out) return fail(MOE_EINVAL, "list is NULL");
  MOE_TRY(need_ptr(host_table, "host_table"));
  if (bytes < grad_table_bytes(count, chunks))
    return fail(MOE_EWORKSPACE, "table of %zu bytes < %zu needed", bytes, grad_table_bytes(count, chunks));
  int a = 0, b = 0;
  if (grad_overlap(list.get(), count, &a, &b)) return fail(MOE_EINVAL, "tensors %d and %d share memory", a, b);
  out->table = nullptr;
  out->count = count;
  out->chunks = grad_table(list.get(), count, host_table);
  return MOE_OK;
}

static moe_status check_grad_call(const moe_grad_list* g, void* ws, size_t ws_bytes, bool needs_ws) {
  if (!g) return fail(MOE_EINVAL, "grads is NULL");
  if (g->count < 0 || g->count > kMaxGrads || g->chunks < 0)
    return fail(MOE_EINVAL, "count=%d / chunks=%d out of range", g->count, g->chunks);
  if (g->chunks > 0) MOE_TRY(need_ptr(g->table, "table"));
  if (!needs_ws) return MOE_OK;
  const size_t need = grad_workspace_bytes();
  if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  return need_ptr(ws, "ws");
}

size_t moe_grad_workspace_bytes(void) { return grad_workspace_bytes(); }

moe_status moe_grad_norm(const moe_grad_list* grads, float* norm, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_grad_call(grads, ws, ws_bytes, true));
  MOE_TRY(need_ptr(norm, "norm"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_GRAD, st, launch_grad_norm(grads->table, grads->count, grads->chunks, norm, ws, st), "gradient norm");
  return MOE_OK;
}

moe_status moe_grad_clip(const moe_grad_list* grads, double max_norm, const float* norm_in, float* norm, void* ws,
                         size_t ws_bytes, void* stream) {
  MOE_TRY(check_grad_call(grads, ws, ws_bytes, !norm_in));
  if (!(max_norm >= 0.0)) return fail(MOE_EINVAL, "max_norm=%g must be >= 0", max_norm);
  MOE_TRY(opt_ptr(norm_in, "norm_in"));
  if (!norm_in) MOE_TRY(need_ptr(norm, "norm"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_GRAD, st,
            launch_grad_clip(grads->table, grads->count, grads->chunks, max_norm, norm_in, norm, ws, st), "gradient clipping");
  return MOE_OK;
}

// ---- 4-bit weights ----
static_assert((int)MOE_W4_INT4 == W4_INT && (int)MOE_W4_FP4 == W4_FP, "format codes");
static_assert((int)MOE_W4_STREAMED == W4_STREAMED && (int)MOE_W4_TILED == W4_TILED && (int)MOE_W4_EXPANDED == W4_EXPANDED, "ways");
static moe_status check_w4_format(int64_t K, int32_t format, int32_t group) {
  if (format != MOE_W4_INT4 && format != MOE_W4_FP4) return fail(MOE_EINVAL, "4-bit format %d invalid", format);
  if (format == MOE_W4_FP4 ? group != 32 : group != 32 && group != 64 && group != 128)
    return fail(MOE_ENOTSUP, "group of %d not supported", group);
  if (K < 1 || K > 65536) return fail(MOE_EINVAL, "K=%lld out of range [1, 65536]", (long long)K);
  if (K % group) return fail(MOE_ENOTSUP, "K=%lld is not a multiple of the group %d", (long long)K, group);
  return MOE_OK;
}
static moe_status check_w4(int64_t K, const moe_w4* w, const char* name, W4View* v) {
  if (!w) return fail(MOE_EINVAL, "%s is NULL", name);
  MOE_TRY(check_w4_format(K, w->format, w->group));
  if (!w->codes || !aligned16(w->codes)) return fail(MOE_EINVAL, "codes of %s are NULL or not 16-byte aligned", name);
  if (!w->scales || !aligned16(w->scales)) return fail(MOE_EINVAL, "scales of %s are NULL or not 16-byte aligned", name);
  *v = W4View{w->codes, w->scales, w->format, w->group};
  return MOE_OK;
}
constexpr int64_t kMaxW4Rows = (int64_t)1 << 31;
static moe_status check_w4_matrix(int64_t rows, int64_t K, int dtype, const moe_w4* w) {
  if (rows < 0 || rows > kMaxW4Rows) return fail(MOE_EINVAL, "rows=%lld out of range [0, 2^31]", (long long)rows);
  if (dtype != MOE_BF16 && dtype != MOE_F32) return fail(MOE_ENOTSUP, "dtype %d not supported", dtype);
  if (!w) return fail(MOE_EINVAL, "w is NULL");
  return check_w4_format(K, w->format, w->group);
}

int64_t moe_w4_scale_bytes(int64_t rows, int64_t K, int32_t format, int32_t group) {
  if (rows < 0 || rows > kMaxW4Rows) return fail(MOE_EINVAL, "rows=%lld out of range [0, 2^31]", (long long)rows), 0;
  if (check_w4_format(K, format, group) != MOE_OK) return 0;
  return format == MOE_W4_INT4 ? K / group * rows * 2 : mx_scale_bytes(rows, K);
}

moe_status moe_quantize_w4(int64_t rows, int64_t K, int dtype, const void* src, const moe_w4* w, void* stream) {
  MOE_TRY(check_w4_matrix(rows, K, dtype, w));
  if (rows == 0) return MOE_OK;
  W4View v;
  MOE_TRY(need_ptr(src, "src"));
  MOE_TRY(check_w4(K, w, "w", &v));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_W4, st, launch_quant_w4(src, dtype == MOE_BF16, v.format, v.group, rows, K, w->codes, w->scales, st),
            "4-bit quantisation");
  return MOE_OK;
}

moe_status moe_dequantize_w4(int64_t rows, int64_t K, int dtype, const moe_w4* w, void* out, void* stream) {
  MOE_TRY(check_w4_matrix(rows, K, dtype, w));
  if (rows == 0) return MOE_OK;
  W4View v;
  MOE_TRY(check_w4(K, w, "w", &v));
  MOE_TRY(need_ptr(out, "out"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_W4, st, launch_expand_w4(v, rows, K, dtype == MOE_BF16, out, st), "4-bit expansion");
  return MOE_OK;
}

moe_status moe_decode_w4(const moe_dims* dims, const void* X, const void* W_r, const float* bias, const moe_w4* W_gate,
                         const moe_w4* W_up, const moe_w4* W_down, float* logits, int32_t* topk_idx, float* topk_w, void* out,
                         void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_dims(dims));
  if (dims->dtype != MOE_BF16) return fail(MOE_ENOTSUP, "4-bit weights need dtype MOE_BF16");
  if (dims->round_mode != MOE_ROUND_NONE)
    return fail(MOE_ENOTSUP, "moe_decode_w4 routes with plain top-K (round_mode must be NONE)");
  if (dims->T > 1024) return fail(MOE_ENOTSUP, "moe_decode_w4 handles T <= 1024 (got %lld)", (long long)dims->T);
  W4View gate, up, down;
  MOE_TRY(check_w4(dims->d, W_gate, "W_gate", &gate));
  MOE_TRY(check_w4(dims->d, W_up, "W_up", &up));
  MOE_TRY(check_w4(dims->n, W_down, "W_down", &down));
  if (up.format != gate.format || up.group != gate.group || down.format != gate.format || down.group != gate.group)
    return fail(MOE_ENOTSUP, "W_gate, W_up and W_down must have one format and group");
  MOE_TRY(need_ptr(X, "X"));
  MOE_TRY(need_ptr(W_r, "W_r"));
  MOE_TRY(opt_ptr(bias, "bias"));
  MOE_TRY(need_ptr(logits, "logits"));
  MOE_TRY(need_ptr(topk_idx, "topk_idx"));
  MOE_TRY(need_ptr(topk_w, "topk_w"));
  MOE_TRY(need_ptr(out, "out"));
  MOE_TRY(check_ws(dims, MOE_OP_DECODE, ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_DECODE, st,
            launch_decode_w4(shape_of(dims), X, W_r, bias, gate, up, down, logits, topk_idx, topk_w, out, ws, st),
            "decode on 4-bit weights");
  return MOE_OK;
}

static moe_status check_linear_w4(const moe_linear_dims* dims, LinShape* s) {
  MOE_TRY(check_linear(dims, s));
  if (!s->bf16) return fail(MOE_ENOTSUP, "4-bit weights need dtype MOE_BF16");
  if (s->K % 32) return fail(MOE_ENOTSUP, "K=%lld must be a multiple of 32", (long long)s->K);
  return MOE_OK;
}

size_t moe_linear_w4_workspace_bytes(const moe_linear_dims* dims) {
  LinShape s;
  return check_linear_w4(dims, &s) == MOE_OK ? linear_w4_workspace_bytes(s) : 0;
}

int moe_linear_w4_plan(const moe_linear_dims* dims) {
  LinShape s;
  MOE_TRY(check_linear_w4(dims, &s));
  return linear_w4_plan(s);
}

int moe_linear_w4_cut(const moe_linear_dims* dims, int32_t* row_tiles, int32_t* token_groups, int32_t* slices) {
  LinShape s;
  MOE_TRY(check_linear_w4(dims, &s));
  const W4Cut c = linear_w4_cut(s);
  if (row_tiles) *row_tiles = c.row_tiles;
  if (token_groups) *token_groups = c.token_groups;
  if (slices) *slices = c.slices;
  return linear_w4_plan(s);
}

moe_status moe_linear_w4(const moe_linear_dims* dims, const void* X, const moe_w4* W, const float* bias,
                         const void* residual, void* out, void* ws, size_t ws_bytes, void* stream) {
  LinShape s;
  MOE_TRY(check_linear_w4(dims, &s));
  if (s.M == 0) return MOE_OK;
  W4View w;
  MOE_TRY(check_w4(s.K, W, "W", &w));
  MOE_TRY(need_ptr(X, "X"));
  MOE_TRY(opt_ptr(bias, "bias"));
  MOE_TRY(opt_ptr(residual, "residual"));
  MOE_TRY(need_ptr(out, "out"));
  MOE_TRY(check_alias(out, s.ldy, residual, s.ldr, "out"));
  if (out == X) return fail(MOE_EINVAL, "out is the X array");
  MOE_TRY(check_linear_ws(linear_w4_workspace_bytes(s), ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_STAGE(MOE_STAGE_LINEAR_W4, st, launch_linear_w4(s, X, w, bias, residual, out, ws, st), "linear on 4-bit weights");
  return MOE_OK;
}

int moe_timing_enable(int on) {
  if (on) {
    if (!g_timing.created) {
      for (int i = 0; i < kTimingSlots; ++i) {
        if (hipEventCreate(&g_timing.ev0[i]) != hipSuccess || hipEventCreate(&g_timing.ev1[i]) != hipSuccess)
          return fail(MOE_EHIP, "hipEventCreate failed");
      }
      g_timing.created = true;
    }
    g_timing.used = 0;
    g_timing.on = true;
    return MOE_OK;
  }
  g_timing.on = false;
  hipError_t first = hipSuccess;
  if (g_timing.created) {
    for (int i = 0; i < g_timing.used; ++i) {
      const hipError_t e = hipEventSynchronize(g_timing.ev1[i]);
      if (first == hipSuccess) first = e;
    }
    for (int i = 0; i < kTimingSlots; ++i) {
      const hipError_t e0 = hipEventDestroy(g_timing.ev0[i]);
      const hipError_t e1 = hipEventDestroy(g_timing.ev1[i]);
      if (first == hipSuccess) first = e0 != hipSuccess ? e0 : e1;
    }
    g_timing.created = false;
  }
  g_timing.used = 0;
  return hip_status(first, "moe_timing_enable(0)");
}

int moe_timing_read(int stage, float* ms, int max) {
  if (stage < 0 || stage >= MOE_STAGE_COUNT) return fail(MOE_EINVAL, "unknown stage %d", stage);
  if (!ms && max > 0) return fail(MOE_EINVAL, "ms is NULL");
  int n = 0;
  for (int i = 0; i < g_timing.used && n < max; ++i) {
    if (g_timing.stage[i] != stage) continue;
    hipError_t e = hipEventSynchronize(g_timing.ev1[i]);
    float t = 0.0f;
    if (e == hipSuccess) e = hipEventElapsedTime(&t, g_timing.ev0[i], g_timing.ev1[i]);
    if (e != hipSuccess) return hip_status(e, "moe_timing_read");
    ms[n++] = t;
  }
  return n;
}

const char* moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "MOE_OK";
    case MOE_EINVAL: return "MOE_EINVAL: invalid argument";
    case MOE_ENOTSUP: return "MOE_ENOTSUP: unsupported shape or dtype";
    case MOE_EWORKSPACE: return "MOE_EWORKSPACE: workspace too small";
    case MOE_EHIP: return "MOE_EHIP: HIP runtime error";
    default: return "unknown moe_status";
  }
}

const char* moe_last_error(void) { return g_err.c_str(); }

const char* moe_version(void) { return "moe_mi355x 0.1 (gfx950)"; }

}  // extern "C"
