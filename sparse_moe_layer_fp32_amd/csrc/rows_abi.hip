// C entry points of the steps between the permutation and the experts' products:
// dispatch, combine, their gradients, and block quantisation.  Declarations and
// the contract are in include/moe.h.

#include "abi_util.h"
#include "rows.h"

namespace {

using moe::check_pointers;
using moe::fail;
using moe::ok;

// A lane takes eight columns, a wave one token's or several tokens' columns, and
// a launch holds fewer than 2^32 threads.
constexpr int64_t kMaxTokens = int64_t(1) << 25;
constexpr int64_t kMaxRows = int64_t(1) << 26;
constexpr int64_t kMaxElements = int64_t(1) << 33;
constexpr int kMaxWidth = 65536;
constexpr int kMaxSlots = 32;

moe_status check_rows(int64_t tokens, int64_t rows, int32_t top_k, int32_t width, const char* name) {
  if (tokens < 0 || rows < 0)
    return fail(MOE_ERR_INVALID_ARG, "negative size (tokens %lld, rows %lld)", (long long)tokens,
                (long long)rows);
  if (top_k < 1 || width < 1)
    return fail(MOE_ERR_INVALID_ARG, "non-positive size (top_k %d, %s %d)", top_k, name, width);
  if (top_k > kMaxSlots) return fail(MOE_ERR_UNSUPPORTED, "top_k %d > %d", top_k, kMaxSlots);
  if (width > kMaxWidth) return fail(MOE_ERR_UNSUPPORTED, "%s %d > %d", name, width, kMaxWidth);
  if (tokens > kMaxTokens || rows > kMaxRows)
    return fail(MOE_ERR_UNSUPPORTED, "%lld tokens > 2^25 or %lld rows > 2^26", (long long)tokens,
                (long long)rows);
  if (tokens * width > kMaxElements || rows * width > kMaxElements)
    return fail(MOE_ERR_UNSUPPORTED, "tokens * %s or rows * %s above 2^33", name, name);
  return MOE_OK;
}

moe_status validate(const moe_dispatch_config* c) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  moe_status st = check_rows(c->tokens, c->rows, c->top_k, c->hidden, "hidden");
  if (st) return st;
  if (c->hidden % 8)
    return fail(MOE_ERR_UNSUPPORTED, "hidden %d not a multiple of 8", c->hidden);
  for (int32_t t : {c->token_dtype, c->row_dtype})
    if (t != MOE_DTYPE_BF16 && t != MOE_DTYPE_F32)
      return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", t);
  return MOE_OK;
}

moe::RowsArgs rows_args(const moe_dispatch_config* c, const int32_t* pair_pos) {
  moe::RowsArgs p{};
  p.tokens = c->tokens;
  p.rows = c->rows;
  p.top_k = c->top_k;
  p.hidden = c->hidden;
  p.pos = pair_pos;
  p.tok_f32 = c->token_dtype == MOE_DTYPE_F32;
  p.row_f32 = c->row_dtype == MOE_DTYPE_F32;
  return p;
}

}  // namespace

extern "C" {

moe_status moe_dispatch_forward(const moe_dispatch_config* cfg, const void* x,
                                const int32_t* pair_pos, void* rows, hipStream_t stream) {
  moe_status st = validate(cfg);
  if (st) return st;
  if (cfg->tokens > 0 && (!x || !pair_pos || (cfg->rows > 0 && !rows)))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_pointers({x, pair_pos, rows}))) return st;
  moe::RowsArgs p = rows_args(cfg, pair_pos);
  p.tok = x;
  p.row_out = rows;
  MOE_CHECK_LAUNCH(moe::launch_dispatch(p, stream), "dispatch");
  return ok();
}

moe_status moe_dispatch_backward(const moe_dispatch_config* cfg, const void* drows,
                                 const int32_t* pair_pos, const void* base, void* dx,
                                 hipStream_t stream) {
  return moe_combine_forward(cfg, drows, pair_pos, nullptr, base, dx, stream);
}

moe_status moe_combine_forward(const moe_dispatch_config* cfg, const void* rows,
                               const int32_t* pair_pos, const float* weights, const void* base,
                               void* y, hipStream_t stream) {
  moe_status st = validate(cfg);
  if (st) return st;
  if (cfg->tokens > 0 && (!pair_pos || !y || (cfg->rows > 0 && !rows)))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_pointers({rows, pair_pos, weights, base, y}))) return st;
  moe::RowsArgs p = rows_args(cfg, pair_pos);
  p.row = rows;
  p.w = weights;
  p.base = base;
  p.tok_out = y;
  MOE_CHECK_LAUNCH(moe::launch_combine_rows(p, stream), "combine");
  return ok();
}

moe_status moe_combine_backward(const moe_dispatch_config* cfg, const void* dy, const void* rows,
                                const int32_t* pair_pos, const float* weights, void* drows,
                                float* dweights, hipStream_t stream) {
  moe_status st = validate(cfg);
  if (st) return st;
  if (cfg->tokens > 0 && (!dy || !pair_pos || (dweights && cfg->rows > 0 && !rows)))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_pointers({dy, rows, pair_pos, weights, drows, dweights}))) return st;
  if (!drows && !dweights) return ok();
  moe::RowsArgs p = rows_args(cfg, pair_pos);
  p.tok = dy;
  p.row = rows;
  p.w = weights;
  p.row_out = drows;
  p.dw = dweights;
  MOE_CHECK_LAUNCH(moe::launch_combine_grad(p, stream), "combine gradient");
  return ok();
}

moe_status moe_quantize_rows(const moe_quantize_config* cfg, const uint16_t* x,
                             const int32_t* pair_pos, uint8_t* codes, float* scales,
                             hipStream_t stream) {
  if (!cfg) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  moe_status st = check_rows(cfg->tokens, cfg->rows, cfg->top_k, cfg->features, "features");
  if (st) return st;
  if (cfg->features % 16)
    return fail(MOE_ERR_UNSUPPORTED, "features %d not a multiple of 16", cfg->features);
  if (!pair_pos && (cfg->rows != cfg->tokens || cfg->top_k != 1) && cfg->tokens > 0)
    return fail(MOE_ERR_INVALID_ARG, "rows %lld, top_k %d without pair_pos (%lld tokens)",
                (long long)cfg->rows, cfg->top_k, (long long)cfg->tokens);
  if (cfg->tokens > 0 && (!x || (cfg->rows > 0 && (!codes || !scales))))
    return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((st = check_pointers({x, pair_pos, codes, scales}))) return st;
  MOE_CHECK_LAUNCH(moe::launch_quantize_rows(x, pair_pos, cfg->tokens, cfg->rows, cfg->top_k,
                                             cfg->features, codes, scales, stream),
                   "quantize rows");
  return ok();
}

moe_status moe_quantize_weight(int32_t num_groups, int32_t out_features, int32_t in_features,
                               const uint16_t* w, uint8_t* codes, float* scales,
                               hipStream_t stream) {
  if (num_groups < 1 || out_features < 1 || in_features < 1)
    return fail(MOE_ERR_INVALID_ARG, "non-positive size (%d x %d x %d)", num_groups, out_features,
                in_features);
  if (in_features % 16)
    return fail(MOE_ERR_UNSUPPORTED, "in_features %d not a multiple of 16", in_features);
  if (out_features > kMaxWidth || in_features > kMaxWidth)
    return fail(MOE_ERR_UNSUPPORTED, "in_features %d / out_features %d > %d", in_features,
                out_features, kMaxWidth);
  const int64_t blocks = static_cast<int64_t>(num_groups) * ((out_features + 127) / 128) *
                         ((in_features + 127) / 128);
  if (blocks > (int64_t(1) << 21))  // 2^35 values in whole blocks
    return fail(MOE_ERR_UNSUPPORTED, "%lld blocks of 128 x 128 > 2^21", (long long)blocks);
  if (!w || !codes || !scales) return fail(MOE_ERR_INVALID_ARG, "a required pointer is NULL");
  moe_status st = check_pointers({w, codes, scales});
  if (st) return st;
  MOE_CHECK_LAUNCH(moe::launch_quantize_weight(w, num_groups, out_features, in_features, codes,
                                               scales, stream),
                   "quantize weight");
  return ok();
}

}  // extern "C"
