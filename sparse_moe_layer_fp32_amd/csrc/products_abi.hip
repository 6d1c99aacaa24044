// C entry points of the linear and grouped products, SwiGLU and their
// gradients: argument validation, workspace layout, launches.  Declarations
// and the contract are in include/moe.h.

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "abi_util.h"
#include "products.h"

namespace {

using moe::align_up;
using moe::aligned16;
using moe::at;
using moe::fail;
using moe::ok;

constexpr int64_t kMaxRows = int64_t(1) << 26;
constexpr int kMaxFeatures = 65536;
constexpr int64_t kMaxElements = int64_t(1) << 35;
constexpr int kMaxGroups = 1024;
// A gathered x is addressed with 32-bit byte offsets, up to this many bytes.
constexpr int64_t kMaxGatherBytes = 0xF0000000ll;

moe_status check_sizes(int64_t rows, int64_t groups, int32_t K, int32_t F) {
  if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows < 0 (%lld)", (long long)rows);
  if (K <= 0 || F <= 0)
    return fail(MOE_ERR_INVALID_ARG, "non-positive size (in_features %d, out_features %d)", K, F);
  if (K % 8 || F % 8)
    return fail(MOE_ERR_UNSUPPORTED, "in_features %d / out_features %d not multiples of 8", K, F);
  if (K > kMaxFeatures || F > kMaxFeatures)
    return fail(MOE_ERR_UNSUPPORTED, "in_features %d / out_features %d > %d", K, F, kMaxFeatures);
  if (rows > kMaxRows)
    return fail(MOE_ERR_UNSUPPORTED, "%lld rows > 2^26", (long long)rows);
  if (rows * std::max(K, F) >= kMaxElements || groups * K * F >= kMaxElements)
    return fail(MOE_ERR_UNSUPPORTED, "rows * features or groups * weights not below 2^35 elements");
  return MOE_OK;
}

moe_status check_dtypes(int32_t y, int32_t dw) {
  for (int32_t t : {y, dw})
    if (t != MOE_DTYPE_BF16 && t != MOE_DTYPE_F32)
      return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", t);
  return MOE_OK;
}

moe_status check_pointers(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (q && !aligned16(q)) return fail(MOE_ERR_UNSUPPORTED, "pointer %p not 16-byte aligned", q);
  return MOE_OK;
}

moe_status check_workspace(size_t need, const void* ws, size_t ws_bytes) {
  if (!need) return MOE_OK;
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned16(ws)) return fail(MOE_ERR_UNSUPPORTED, "workspace not 16-byte aligned");
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  return MOE_OK;
}

// Compute units of the current device, looked up once per device; an
// MI355X's 256 where there is none (a workspace can be sized on a host
// without a GPU).
int device_cus() {
  static std::atomic<int> known[64];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return 256;
  }
  const bool slot = dev >= 0 && dev < 64;
  if (slot && (cus = known[dev].load(std::memory_order_relaxed)) > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      cus <= 0) {
    (void)hipGetLastError();
    return 256;
  }
  if (slot) known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

// The plans of a map's three products, and its workspace: source rows (the
// gathered weight gradient), then one area that the products use in turn
// (partial sums, strip sums).
struct MapPlan {
  int64_t P;
  int G, K, F;
  moe::ProductPlan fwd, dx, dw;
  size_t src, part, total;
};

void make_map_plan(int64_t P, int G, int K, int F, bool grouped, MapPlan* m) {
  m->P = P;
  m->G = G;
  m->K = K;
  m->F = F;
  const int cus = device_cus();
  m->fwd = moe::product_plan(moe::kForward, P, G, K, F, cus);
  m->dx = moe::product_plan(moe::kInputGrad, P, G, K, F, cus);
  m->dw = moe::product_plan(moe::kWeightGrad, P, G, K, F, cus);
  size_t part = std::max({moe::product_part_bytes(moe::kForward, P, G, K, F, m->fwd),
                          moe::product_part_bytes(moe::kInputGrad, P, G, K, F, m->dx),
                          moe::product_part_bytes(moe::kWeightGrad, P, G, K, F, m->dw)});
  if (!grouped) part = std::max(part, moe::act_grad_part_bytes(P, F));
  m->src = 0;
  m->part = grouped ? align_up((static_cast<size_t>(P) + moe::kSourcePad) * 4) : 0;
  m->total = std::max<size_t>(m->part + align_up(part), moe::kAlign);
}

moe_status validate_linear(const moe_linear_config* c) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  moe_status st = check_sizes(c->tokens, 1, c->in_features, c->out_features);
  if (st) return st;
  if (c->activation < MOE_ACT_NONE || c->activation > MOE_ACT_SILU)
    return fail(MOE_ERR_INVALID_ARG, "unknown activation %d", c->activation);
  return check_dtypes(c->y_dtype, c->dw_dtype);
}

moe_status validate_grouped(const moe_grouped_config* c) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  if (c->num_groups < 1)
    return fail(MOE_ERR_INVALID_ARG, "num_groups %d < 1", c->num_groups);
  if (c->num_groups > kMaxGroups)
    return fail(MOE_ERR_UNSUPPORTED, "num_groups %d > %d", c->num_groups, kMaxGroups);
  moe_status st = check_sizes(c->rows, c->num_groups, c->in_features, c->out_features);
  if (st) return st;
  if (c->row_div < 1) return fail(MOE_ERR_INVALID_ARG, "row_div %d < 1", c->row_div);
  if (c->x_rows < 0) return fail(MOE_ERR_INVALID_ARG, "x_rows < 0 (%lld)", (long long)c->x_rows);
  if (c->reserved) return fail(MOE_ERR_INVALID_ARG, "reserved field must be 0");
  return check_dtypes(c->y_dtype, c->dw_dtype);
}

// x behind row_ids, or by itself.
moe_status check_gather(const moe_grouped_config* c, const int32_t* row_ids) {
  if (c->rows == 0) return MOE_OK;  // row_ids has no entries
  if (!row_ids && c->x_rows != c->rows)
    return fail(MOE_ERR_INVALID_ARG, "x_rows %lld differs from rows %lld without row_ids",
                (long long)c->x_rows, (long long)c->rows);
  if (row_ids && (c->x_rows > kMaxRows || c->x_rows * c->in_features * 2 >= kMaxGatherBytes))
    return fail(MOE_ERR_UNSUPPORTED, "x_rows * in_features must be below %lld with row_ids",
                (long long)(kMaxGatherBytes / 2));
  return MOE_OK;
}

moe_status validate_swiglu(const moe_swiglu_config* c, int64_t* ld) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  if (c->rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows < 0 (%lld)", (long long)c->rows);
  if (c->inter <= 0) return fail(MOE_ERR_INVALID_ARG, "non-positive size (inter %d)", c->inter);
  if (c->reserved) return fail(MOE_ERR_INVALID_ARG, "reserved field must be 0");
  *ld = c->ld ? c->ld : c->inter;
  if (*ld < c->inter)
    return fail(MOE_ERR_INVALID_ARG, "row stride %d < inter %d", c->ld, c->inter);
  if (c->inter % 8 || *ld % 8)
    return fail(MOE_ERR_UNSUPPORTED, "inter %d / row stride %d not multiples of 8", c->inter,
                static_cast<int>(*ld));
  // (a thread takes 8 elements, and a launch, in blocks of 256, holds fewer than 2^32 threads)
  if (c->rows > (kMaxElements - 2048) / *ld)
    return fail(MOE_ERR_UNSUPPORTED, "rows * row stride above 2^35 - 2048 elements");
  return MOE_OK;
}

moe::ProductArgs map_args(const MapPlan& m, void* ws) {
  moe::ProductArgs p{};
  p.row_div = 1;
  p.x_rows = m.P;
  p.P = m.P;
  p.G = m.G;
  p.K = m.K;
  p.F = m.F;
  p.part = ws ? at<float>(ws, m.part) : nullptr;
  return p;
}

// The input and weight gradients that are wanted of p (with a = dy).
hipError_t gradients(const MapPlan& m, const moe::ProductArgs& p, const uint16_t* w,
                     const uint16_t* x, uint16_t* dx, void* dw, float* db, bool dw_f32,
                     bool accumulate, const int32_t* src, int64_t x_rows, hipStream_t stream) {
  moe::ProductArgs px = p, pw = p;
  px.b = w;
  px.y = dx;
  pw.b = x;
  pw.y = dw;
  pw.y_f32 = dw_f32;
  pw.accumulate = accumulate;
  pw.db = db;
  pw.src = src;
  pw.x_rows = x_rows;
  const bool want_w = dw || db;
  moe::ProductPlan plan_x, plan_w;
  if (dx && dw && moe::pair_plan(m.P, m.G, m.K, m.F, m.dx.cus, &plan_x, &plan_w))
    return moe::launch_pair(px, plan_x, pw, plan_w, stream);
  hipError_t e = hipSuccess;
  if (dx) e = moe::launch_product(moe::kInputGrad, px, m.dx, stream);
  if (e == hipSuccess && want_w) e = moe::launch_product(moe::kWeightGrad, pw, m.dw, stream);
  return e;
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(const moe_linear_config* cfg) {
  if (validate_linear(cfg) != MOE_OK) return 0;
  MapPlan m;
  make_map_plan(cfg->tokens, 1, cfg->in_features, cfg->out_features, false, &m);
  return m.total;
}

moe_status moe_linear_forward(const moe_linear_config* cfg, const uint16_t* x, const uint16_t* w,
                              const float* bias, const uint16_t* residual, void* y, uint16_t* z,
                              void* ws, size_t ws_bytes, hipStream_t stream) {
  moe_status st = validate_linear(cfg);
  if (st) return st;
  if (!w || (cfg->tokens > 0 && (!x || !y)))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_pointers({x, w, bias, residual, y, z}))) return st;
  MapPlan m;
  make_map_plan(cfg->tokens, 1, cfg->in_features, cfg->out_features, false, &m);
  if ((st = check_workspace(m.total, ws, ws_bytes))) return st;
  if (cfg->tokens == 0) return ok();
  moe::ProductArgs p = map_args(m, ws);
  p.a = x;
  p.b = w;
  p.bias = bias;
  p.residual = residual;
  p.z = z;
  p.y = y;
  p.y_f32 = cfg->y_dtype == MOE_DTYPE_F32;
  p.act = cfg->activation;
  MOE_CHECK_LAUNCH(moe::launch_product(moe::kForward, p, m.fwd, stream), "linear forward");
  return ok();
}

moe_status moe_linear_backward(const moe_linear_config* cfg, const uint16_t* dy, const uint16_t* z,
                               const uint16_t* x, const uint16_t* w, uint16_t* dz, uint16_t* dx,
                               void* dw, float* dbias, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
  moe_status st = validate_linear(cfg);
  if (st) return st;
  const bool act = cfg->activation != MOE_ACT_NONE;
  if (cfg->tokens > 0 && (!dy || (act && (!z || !dz)) || (dx && !w) || (dw && !x)))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_pointers({dy, z, x, w, dz, dx, dw, dbias}))) return st;
  MapPlan m;
  make_map_plan(cfg->tokens, 1, cfg->in_features, cfg->out_features, false, &m);
  if ((st = check_workspace(m.total, ws, ws_bytes))) return st;
  moe::ProductArgs p = map_args(m, ws);
  p.a = dy;
  if (act && cfg->tokens > 0) {
    MOE_CHECK_LAUNCH(moe::launch_act_grad(dy, z, cfg->activation, m.P, m.F, dz, dbias,
                                          cfg->accumulate != 0, p.part, stream),
                     "activation gradient");
    p.a = dz;
  }
  // dbias with an activation is done above, except that nothing ran for 0 tokens
  float* db = act && cfg->tokens > 0 ? nullptr : dbias;
  MOE_CHECK_LAUNCH(gradients(m, p, w, x, cfg->tokens > 0 ? dx : nullptr, dw, db,
                             cfg->dw_dtype == MOE_DTYPE_F32, cfg->accumulate != 0, nullptr, m.P, stream),
                   "linear gradients");
  return ok();
}

size_t moe_grouped_workspace_size(const moe_grouped_config* cfg) {
  if (validate_grouped(cfg) != MOE_OK) return 0;
  MapPlan m;
  make_map_plan(cfg->rows, cfg->num_groups, cfg->in_features, cfg->out_features, true, &m);
  return m.total;
}

moe_status moe_grouped_forward(const moe_grouped_config* cfg, const uint16_t* x,
                               const int32_t* row_ids, const int32_t* offsets, const uint16_t* w,
                               const float* bias, void* y, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
  moe_status st = validate_grouped(cfg);
  if (st) return st;
  if (!offsets || !w || (cfg->rows > 0 && ((cfg->x_rows > 0 && !x) || !y)))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_gather(cfg, row_ids))) return st;
  if ((st = check_pointers({x, row_ids, offsets, w, bias, y}))) return st;
  MapPlan m;
  make_map_plan(cfg->rows, cfg->num_groups, cfg->in_features, cfg->out_features, true, &m);
  if ((st = check_workspace(m.total, ws, ws_bytes))) return st;
  if (cfg->rows == 0) return ok();
  moe::ProductArgs p = map_args(m, ws);
  p.a = x;
  p.b = w;
  p.offsets = offsets;
  p.src = row_ids;
  p.row_div = cfg->row_div;
  p.x_rows = cfg->x_rows;
  p.bias = bias;
  p.y = y;
  p.y_f32 = cfg->y_dtype == MOE_DTYPE_F32;
  MOE_CHECK_LAUNCH(moe::launch_product(moe::kForward, p, m.fwd, stream), "grouped forward");
  return ok();
}

moe_status moe_grouped_backward(const moe_grouped_config* cfg, const uint16_t* dy,
                                const uint16_t* x, const int32_t* row_ids, const int32_t* offsets,
                                const uint16_t* w, uint16_t* dx, void* dw, float* dbias, void* ws,
                                size_t ws_bytes, hipStream_t stream) {
  moe_status st = validate_grouped(cfg);
  if (st) return st;
  if (!offsets ||
      (cfg->rows > 0 && (!dy || (dx && !w) || (dw && cfg->x_rows > 0 && !x))))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if (dw && (st = check_gather(cfg, row_ids))) return st;
  if ((st = check_pointers({dy, x, row_ids, offsets, w, dx, dw, dbias}))) return st;
  MapPlan m;
  make_map_plan(cfg->rows, cfg->num_groups, cfg->in_features, cfg->out_features, true, &m);
  if ((st = check_workspace(m.total, ws, ws_bytes))) return st;
  moe::ProductArgs p = map_args(m, ws);
  p.a = dy;
  p.offsets = offsets;
  const bool gather = dw && row_ids && cfg->rows > 0;
  int32_t* src = gather ? at<int32_t>(ws, m.src) : nullptr;
  if (gather)
    MOE_CHECK_LAUNCH(moe::launch_source_rows(row_ids, cfg->row_div, cfg->x_rows, m.P, src, stream),
                     "source rows");
  MOE_CHECK_LAUNCH(gradients(m, p, w, x, cfg->rows > 0 ? dx : nullptr, dw, dbias,
                             cfg->dw_dtype == MOE_DTYPE_F32, cfg->accumulate != 0, src,
                             gather ? cfg->x_rows : m.P, stream),
                   "grouped gradients");
  return ok();
}

moe_status moe_swiglu_forward(const moe_swiglu_config* cfg, const uint16_t* gate,
                              const uint16_t* up, uint16_t* h, hipStream_t stream) {
  int64_t ld = 0;
  moe_status st = validate_swiglu(cfg, &ld);
  if (st) return st;
  if (cfg->rows > 0 && (!gate || !up || !h))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_pointers({gate, up, h}))) return st;
  MOE_CHECK_LAUNCH(moe::launch_swiglu(gate, up, h, cfg->rows, cfg->inter, ld, cfg->limit, stream),
                   "swiglu");
  return ok();
}

moe_status moe_swiglu_backward(const moe_swiglu_config* cfg, const uint16_t* dh,
                               const uint16_t* gate, const uint16_t* up, uint16_t* dgate,
                               uint16_t* dup, uint16_t* h, hipStream_t stream) {
  int64_t ld = 0;
  moe_status st = validate_swiglu(cfg, &ld);
  if (st) return st;
  if (cfg->rows > 0 && (!dh || !gate || !up || !dgate || !dup))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_pointers({dh, gate, up, dgate, dup, h}))) return st;
  MOE_CHECK_LAUNCH(moe::launch_swiglu_grad(dh, gate, up, dgate, dup, h, cfg->rows, cfg->inter, ld,
                                           cfg->limit, stream),
                   "swiglu gradient");
  return ok();
}

}  // extern "C"
