// C ABI of what surrounds the layer: the norm, the dropout with the residual
// sum, and the products and experts with 4-bit weights.  Argument checks and
// workspace carve-up, as in capi.cu.
#include <math.h>

#include "common.cuh"

namespace {

using namespace moe;

#define MOE_TRY(expr)                      \
  do {                                     \
    const moe_status st_ = (expr);         \
    if (st_ != MOE_OK) return st_;         \
  } while (0)
#define MOE_CUDA(expr) MOE_TRY(cuda_status(expr))

moe_status need(const void* p, uint64_t nelem, size_t align = 16) {
  if (nelem == 0) return MOE_OK;
  return p == nullptr || reinterpret_cast<uintptr_t>(p) % align != 0 ? MOE_ERR_INVALID_ARG
                                                                     : MOE_OK;
}
moe_status optional(const void* p, size_t align = 16) {
  return reinterpret_cast<uintptr_t>(p) % align != 0 ? MOE_ERR_INVALID_ARG : MOE_OK;
}
moe_status check_ws(const void* ws, size_t have, size_t want) {
  if (ws == nullptr || reinterpret_cast<uintptr_t>(ws) % 16 != 0) return MOE_ERR_INVALID_ARG;
  return have < want ? MOE_ERR_WORKSPACE : MOE_OK;
}
void* past_error_word(void* ws) { return static_cast<char*>(ws) + kErrBytes; }

bool is_dtype(int32_t d) { return d == MOE_F32 || d == MOE_BF16; }
bool is_probability(double p) { return p >= 0.0 && p <= 1.0; }  // false for NaN

// Elements of one tensor: 2^46 bf16 values are past any device's memory.
constexpr int64_t kMaxElements = int64_t{1} << 46;

moe_status validate(const moe_norm_config* c) {
  if (c == nullptr || c->rows < 0 || c->hidden <= 0) return MOE_ERR_INVALID_ARG;
  if (!is_dtype(c->dtype) || !is_dtype(c->param_dtype)) return MOE_ERR_INVALID_ARG;
  if (c->kind != MOE_NORM_LAYER && c->kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARG;
  if (!is_probability(c->dropout)) return MOE_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || isinf(c->eps)) return MOE_ERR_INVALID_ARG;
  if (c->dtype == MOE_F32 && c->param_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (c->hidden > (1 << 24) || c->rows > kMaxElements / c->hidden) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t norm_backward_bytes(const moe_norm_config& c, int ctas) {
  return kErrBytes + static_cast<size_t>(ctas) * 2 * c.hidden * 4;
}

bool is_group(int32_t g) { return g == 32 || g == 64 || g == 128; }

// A 4-bit weight of [rows, K]
moe_status need_w4(const moe_w4* w, uint64_t rows, W4* out) {
  if (w == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(need(w->codes, rows));
  MOE_TRY(need(w->scales, rows));
  MOE_TRY(optional(w->zeros));
  *out = {w->codes, static_cast<const __nv_bfloat16*>(w->scales), w->zeros};
  return MOE_OK;
}

moe_status validate_linear(int64_t rows, int32_t N, int32_t K) {
  if (rows < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (K % 32 != 0) return MOE_ERR_UNSUPPORTED;
  if (rows > (int64_t{1} << 30) || N > (1 << 28) || K > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The layer's own checks of the configuration, then those of the 4-bit experts.
moe_status validate_experts(const moe_config* cfg) {
  size_t bytes = 0;
  MOE_TRY(moe_workspace_size(cfg, &bytes));
  // rows of a weight, over all experts, are counted in 32 bits
  const int64_t most = (int64_t{1} << 31) / cfg->num_experts;
  if (cfg->hidden >= most || cfg->ffn_hidden >= most) return MOE_ERR_UNSUPPORTED;
  return cfg->dtype == MOE_BF16 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// most: what any call of up to that many tokens needs, not this one alone
size_t experts_bytes(const moe_config& c, bool most) {
  return kErrBytes +
         (most ? w4_experts_scratch_most : w4_experts_scratch)(c.num_tokens, c.hidden,
                                                               c.num_experts, c.topk, c.ffn_hidden);
}

// moe_forward_w4: the layer's workspace (moe_route's, with the error word),
// the routing outputs, then the experts' workspace.
struct ForwardLayout {
  size_t idx, prob, keep, tpe, experts, total;
};
moe_status forward_layout(const moe_config& c, bool most, ForwardLayout* L) {
  size_t o = 0;
  MOE_TRY(moe_workspace_size(&c, &o));
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o = (o + bytes + 255) & ~static_cast<size_t>(255);
    return r;
  };
  const size_t pairs = static_cast<size_t>(c.num_tokens) * c.topk;
  L->idx = take(pairs * 4);
  L->prob = take(pairs * 4);
  L->keep = take(pairs);
  L->tpe = take(static_cast<size_t>(c.num_experts) * 4);
  L->experts = take(experts_bytes(c, most) - kErrBytes);
  L->total = o;
  return MOE_OK;
}

moe_status experts_checks(const moe_config& c, int32_t group, const moe_w4* W1, const moe_w4* W3,
                          const moe_w4* W2, W4* w1, W4* w3, W4* w2) {
  if (!is_group(group)) return MOE_ERR_INVALID_ARG;
  const uint64_t E = c.num_experts;
  MOE_TRY(need_w4(W1, E * c.ffn_hidden, w1));
  MOE_TRY(need_w4(W3, E * c.ffn_hidden, w3));
  MOE_TRY(need_w4(W2, E * c.hidden, w2));
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_layer_norm(const moe_norm_config* cfg, const void* x, const void* residual,
                          const uint64_t* rng, const void* weight, const void* bias, void* z,
                          void* y, float* mean, float* rstd, moe_stream_t stream) {
  MOE_TRY(validate(cfg));
  const moe_norm_config& c = *cfg;
  const uint64_t n = static_cast<uint64_t>(c.rows) * c.hidden;
  MOE_TRY(need(x, n));
  MOE_TRY(need(y, n));
  MOE_TRY(optional(residual));
  MOE_TRY(optional(z));
  MOE_TRY(optional(weight));
  MOE_TRY(optional(bias));
  MOE_TRY(optional(mean));
  MOE_TRY(optional(rstd));
  if (n > 0 && residual == nullptr && (z != nullptr || c.dropout > 0.0))
    return MOE_ERR_INVALID_ARG;
  if (n > 0 && z == y) return MOE_ERR_INVALID_ARG;
  if (c.dropout > 0.0) MOE_TRY(need(rng, n));
  MOE_CUDA(launch_norm(c, x, residual, rng, weight, bias, z, y, mean, rstd, stream));
  return MOE_OK;
}

moe_status moe_workspace_size_norm_backward(const moe_norm_config* cfg, size_t* bytes) {
  MOE_TRY(validate(cfg));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = norm_backward_bytes(*cfg, norm_backward_ctas_most(*cfg));
  return MOE_OK;
}

moe_status moe_layer_norm_backward(const moe_norm_config* cfg, const void* dy, const void* z,
                                   const void* weight, const float* mean, const float* rstd,
                                   const void* dz, const uint64_t* rng, void* dx, void* dbranch,
                                   float* dweight, float* dbias, void* ws, size_t ws_bytes,
                                   moe_stream_t stream) {
  MOE_TRY(validate(cfg));
  const moe_norm_config& c = *cfg;
  const uint64_t n = static_cast<uint64_t>(c.rows) * c.hidden;
  MOE_TRY(need(dy, n));
  MOE_TRY(need(z, n));
  MOE_TRY(need(dx, n));
  MOE_TRY(need(rstd, static_cast<uint64_t>(c.rows)));
  if (c.kind == MOE_NORM_LAYER) MOE_TRY(need(mean, static_cast<uint64_t>(c.rows)));
  MOE_TRY(optional(weight));
  MOE_TRY(optional(dz));
  MOE_TRY(optional(dbranch));
  MOE_TRY(optional(dweight));
  MOE_TRY(optional(dbias));
  if (dbranch != nullptr && dbranch == dx) return MOE_ERR_INVALID_ARG;
  if (dbranch != nullptr && c.dropout > 0.0) MOE_TRY(need(rng, n));
  MOE_TRY(check_ws(ws, ws_bytes, norm_backward_bytes(c, norm_backward_ctas(c))));
  MOE_CUDA(launch_norm_backward(c, dy, z, weight, mean, rstd, dz, rng, dx, dbranch, dweight,
                                dbias, static_cast<float*>(past_error_word(ws)), stream));
  return MOE_OK;
}

moe_status moe_dropout_add(int64_t n, int32_t dtype, double dropout, const uint64_t* rng,
                           const void* x, const void* residual, void* y, moe_stream_t stream) {
  if (n < 0 || !is_dtype(dtype) || !is_probability(dropout)) return MOE_ERR_INVALID_ARG;
  if (n > kMaxElements) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(need(x, n));
  MOE_TRY(need(y, n));
  MOE_TRY(optional(residual));
  if (dropout > 0.0) MOE_TRY(need(rng, n));
  MOE_CUDA(launch_dropout_add(n, dtype, dropout, rng, x, residual, y, stream));
  return MOE_OK;
}

moe_status moe_quantize_w4(int32_t experts, int32_t K, int32_t N, int32_t group, const void* W,
                           uint8_t* codes, void* scales, uint8_t* zeros, moe_stream_t stream) {
  if (experts <= 0 || K <= 0 || N <= 0 || !is_group(group)) return MOE_ERR_INVALID_ARG;
  if (K % 64 != 0 || N % 64 != 0 || K % group != 0 || experts > 65535 || K / group > 65535)
    return MOE_ERR_UNSUPPORTED;
  MOE_TRY(need(W, 1));
  MOE_TRY(need(codes, 1));
  MOE_TRY(need(scales, 1));
  MOE_TRY(optional(zeros));
  MOE_CUDA(launch_w4_quantize(experts, K, N, group, W, codes, scales, zeros, stream));
  return MOE_OK;
}

moe_status moe_pack_w4(int32_t experts, int32_t N, int32_t K, const uint8_t* values,
                       uint8_t* codes, moe_stream_t stream) {
  if (experts <= 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  MOE_TRY(need(values, 1));
  MOE_TRY(need(codes, 1));
  MOE_CUDA(launch_w4_pack(experts, N, K, values, codes, stream));
  return MOE_OK;
}

moe_status moe_workspace_size_linear_w4(int64_t rows, int32_t N, int32_t K, size_t* bytes) {
  MOE_TRY(validate_linear(rows, N, K));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = kErrBytes + w4_linear_scratch_most(rows, N, K);
  return MOE_OK;
}

moe_status moe_linear_w4(int64_t rows, int32_t N, int32_t K, int32_t group, const void* x,
                         const moe_w4* W, void* y, int32_t y_dtype, void* ws, size_t ws_bytes,
                         moe_stream_t stream) {
  MOE_TRY(validate_linear(rows, N, K));
  if (!is_group(group) || !is_dtype(y_dtype)) return MOE_ERR_INVALID_ARG;
  if (K % group != 0) return MOE_ERR_UNSUPPORTED;
  W4 w;
  MOE_TRY(need_w4(W, N, &w));
  MOE_TRY(need(x, rows));
  MOE_TRY(need(y, rows));
  MOE_TRY(check_ws(ws, ws_bytes, kErrBytes + w4_linear_scratch(rows, N, K)));
  if (rows == 0) return MOE_OK;
  MOE_CUDA(launch_w4_linear(rows, N, K, group, x, w, y, y_dtype, past_error_word(ws),
                            static_cast<int*>(ws), stream));
  return MOE_OK;
}

moe_status moe_workspace_size_experts_w4(const moe_config* cfg, size_t* bytes) {
  MOE_TRY(validate_experts(cfg));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = experts_bytes(*cfg, true);
  return MOE_OK;
}

moe_status moe_experts_w4(const moe_config* cfg, int32_t group, const void* x,
                          const int32_t* topk_idx, const float* topk_prob, const uint8_t* keep,
                          const moe_w4* W1, const moe_w4* W3, const moe_w4* W2, void* y, void* ws,
                          size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(validate_experts(cfg));
  const moe_config& c = *cfg;
  W4 w1, w3, w2;
  MOE_TRY(experts_checks(c, group, W1, W3, W2, &w1, &w3, &w2));
  const uint64_t T = c.num_tokens;
  MOE_TRY(need(x, T));
  MOE_TRY(need(topk_idx, T, 4));
  MOE_TRY(need(topk_prob, T, 4));
  MOE_TRY(need(y, T));
  MOE_TRY(check_ws(ws, ws_bytes, experts_bytes(c, false)));
  if (T == 0) return MOE_OK;
  MOE_CUDA(launch_w4_experts(c.num_tokens, c.hidden, c.num_experts, c.topk, c.ffn_hidden, group, x,
                             topk_idx, topk_prob, keep, w1, w3, w2, y, past_error_word(ws),
                             static_cast<int*>(ws), stream));
  return MOE_OK;
}

moe_status moe_workspace_size_w4(const moe_config* cfg, size_t* bytes) {
  MOE_TRY(validate_experts(cfg));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  ForwardLayout L;
  MOE_TRY(forward_layout(*cfg, true, &L));
  *bytes = L.total;
  return MOE_OK;
}

moe_status moe_forward_w4(const moe_config* cfg, int32_t group, const void* x, const float* Wg,
                          const float* gate_bias, const float* expert_bias, const moe_w4* W1,
                          const moe_w4* W3, const moe_w4* W2, void* y, int32_t* topk_idx,
                          float* topk_prob, int32_t* tokens_per_expert, void* ws,
                          size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(validate_experts(cfg));
  moe_config c = *cfg;
  W4 w1, w3, w2;
  MOE_TRY(experts_checks(c, group, W1, W3, W2, &w1, &w3, &w2));
  const uint64_t T = c.num_tokens;
  MOE_TRY(need(x, T));
  MOE_TRY(need(Wg, 1, 4));
  MOE_TRY(optional(gate_bias, 4));
  MOE_TRY(optional(expert_bias, 4));
  MOE_TRY(need(y, T));
  MOE_TRY(optional(topk_idx, 4));
  MOE_TRY(optional(topk_prob, 4));
  MOE_TRY(optional(tokens_per_expert, 4));
  ForwardLayout L;
  MOE_TRY(forward_layout(c, false, &L));
  MOE_TRY(check_ws(ws, ws_bytes, L.total));
  char* base = static_cast<char*>(ws);
  int32_t* idx = topk_idx ? topk_idx : reinterpret_cast<int32_t*>(base + L.idx);
  float* prob = topk_prob ? topk_prob : reinterpret_cast<float*>(base + L.prob);
  int32_t* tpe = tokens_per_expert ? tokens_per_expert : reinterpret_cast<int32_t*>(base + L.tpe);
  uint8_t* keep = reinterpret_cast<uint8_t*>(base + L.keep);
  c.pad_to_capacity = 0;
  MOE_TRY(moe_route(&c, x, Wg, gate_bias, expert_bias, idx, prob, keep, tpe, nullptr, ws, ws_bytes,
                    stream));
  if (T == 0) return MOE_OK;
  MOE_CUDA(launch_w4_experts(c.num_tokens, c.hidden, c.num_experts, c.topk, c.ffn_hidden, group, x,
                             idx, prob, keep, w1, w3, w2, y, base + L.experts,
                             static_cast<int*>(ws), stream));
  return MOE_OK;
}

}  // extern "C"
