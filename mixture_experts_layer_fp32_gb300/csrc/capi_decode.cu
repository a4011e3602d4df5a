// C ABI of a decoding step: the whole layer for a few tokens, the choice of the next
// token, products in 8-bit integers.  Argument checks and workspace carve-up, as in
// capi.cu.
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

// The layer's own checks of the configuration, then those of few tokens.
moe_status validate_few(const moe_config* cfg, int32_t fs) {
  size_t bytes = 0;
  MOE_TRY(moe_workspace_size(cfg, &bytes));
  if (fs < 0) return MOE_ERR_INVALID_ARG;
  if (fs % (cfg->dtype == MOE_BF16 ? 128 : 8) != 0) return MOE_ERR_UNSUPPORTED;
  if (cfg->num_tokens > MOE_FEW_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
  // a row's inputs and all rows' inputs are counted in 32 bits
  constexpr int32_t most = 1 << 21;
  if (cfg->hidden > most || cfg->ffn_hidden > most || fs > most) return MOE_ERR_UNSUPPORTED;
  // the weights of one kind are counted in units in 32 bits: 16 inputs of 512 outputs (of
  // FC1, 256 of W1 and the same of W3) or more, here taken as 16 x 256
  auto units = [](int64_t in, int64_t out) { return (in + 15) / 16 * ((out + 255) / 256); };
  const int64_t h = cfg->hidden, f = cfg->ffn_hidden;
  const int64_t up = cfg->num_experts * units(h, f) + units(h, fs);
  const int64_t down = cfg->num_experts * units(f, h) + units(fs, h);
  if (up >= int64_t{1} << 31 || down >= int64_t{1} << 31) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status validate_i8(int64_t rows, int32_t N, int32_t K) {
  if (rows < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > 131056 || N > (1 << 28) || rows > (1 << 28)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_workspace_size_few(const moe_config* cfg, int32_t fs, size_t* bytes) {
  MOE_TRY(validate_few(cfg, fs));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = kErrBytes + few_scratch(*cfg, fs);
  return MOE_OK;
}

moe_status moe_forward_few(const moe_config* cfg, int32_t fs, const void* x, const float* Wg,
                           const float* gate_bias, const float* expert_bias, const void* W1,
                           const void* W3, const void* W2, const void* W1s, const void* W3s,
                           const void* W2s, void* y, int32_t* topk_idx, float* topk_prob,
                           int32_t* tokens_per_expert, void* ws, size_t ws_bytes,
                           moe_stream_t stream) {
  MOE_TRY(validate_few(cfg, fs));
  const uint64_t T = cfg->num_tokens;
  MOE_TRY(need(x, T));
  MOE_TRY(need(Wg, 1));
  MOE_TRY(optional(gate_bias, 4));
  MOE_TRY(optional(expert_bias, 4));
  MOE_TRY(need(W1, 1));
  MOE_TRY(need(W3, 1));
  MOE_TRY(need(W2, 1));
  MOE_TRY(need(W1s, fs));
  MOE_TRY(need(W3s, fs));
  MOE_TRY(need(W2s, fs));
  MOE_TRY(need(y, T));
  MOE_TRY(optional(topk_idx, 4));
  MOE_TRY(optional(topk_prob, 4));
  MOE_TRY(optional(tokens_per_expert, 4));
  MOE_TRY(check_ws(ws, ws_bytes, kErrBytes + few_scratch(*cfg, fs)));
  int64_t capacity = -1;
  MOE_TRY(moe_capacity(cfg, &capacity));
  if (T == 0) {
    if (tokens_per_expert != nullptr)
      MOE_CUDA(cudaMemsetAsync(tokens_per_expert, 0, sizeof(int32_t) * cfg->num_experts, stream));
    return MOE_OK;
  }
  MOE_CUDA(launch_few(*cfg, fs, capacity, x, Wg, gate_bias, expert_bias, W1, W3, W2, W1s, W3s, W2s,
                      y, topk_idx, topk_prob, tokens_per_expert, past_error_word(ws),
                      static_cast<int*>(ws), stream));
  return MOE_OK;
}

moe_status moe_sample(int64_t rows, int32_t vocab, int32_t dtype, const void* logits,
                      const float* u, const moe_sample_choices* choices, int32_t* tokens,
                      float* prob, moe_stream_t stream) {
  if (rows < 0 || vocab <= 0 || choices == nullptr || !is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  // sums of weights of up to 2^40 are held in 64 bits
  if (vocab >= (1 << 24) || rows >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED;
  const moe_sample_choices& c = *choices;
  // false for NaN
  if (!(c.temperature >= 0.f) || c.top_k < 0 || !(c.top_p >= 0.f && c.top_p <= 1.f) ||
      !(c.min_p >= 0.f && c.min_p <= 1.f))
    return MOE_ERR_INVALID_ARG;
  const uint64_t n = rows;
  MOE_TRY(need(logits, n));
  MOE_TRY(need(u, n, 4));
  MOE_TRY(need(tokens, n, 4));
  MOE_TRY(optional(prob, 4));
  MOE_TRY(optional(c.temperature_of, 4));
  MOE_TRY(optional(c.top_k_of, 4));
  MOE_TRY(optional(c.top_p_of, 4));
  MOE_TRY(optional(c.min_p_of, 4));
  if (rows == 0) return MOE_OK;
  const SampleChoices own = {c.temperature,    c.top_k,    c.top_p,    c.min_p,
                             c.temperature_of, c.top_k_of, c.top_p_of, c.min_p_of};
  MOE_CUDA(launch_sample(rows, vocab, dtype, logits, u, own, tokens, prob, stream));
  return MOE_OK;
}

moe_status moe_quantize_rows_i8(int64_t rows, int32_t K, int32_t dtype, const void* x,
                                int8_t* codes, float* scales, moe_stream_t stream) {
  MOE_TRY(validate_i8(rows, 1, K));
  if (!is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(need(x, rows));
  MOE_TRY(need(codes, rows));
  MOE_TRY(need(scales, rows, 4));
  if (rows == 0) return MOE_OK;
  MOE_CUDA(launch_quantize_rows_i8(rows, K, dtype, x, codes, scales, stream));
  return MOE_OK;
}

moe_status moe_workspace_size_linear_i8(int64_t rows, int32_t N, int32_t K, size_t* bytes) {
  MOE_TRY(validate_i8(rows, N, K));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = kErrBytes + i8_linear_scratch_most(rows, N, K);
  return MOE_OK;
}

moe_status moe_linear_i8(int64_t rows, int32_t N, int32_t K, const void* x, int32_t x_dtype,
                         const float* x_scale, const int8_t* W, const float* w_scale,
                         const float* bias, void* y, int32_t y_dtype, void* ws, size_t ws_bytes,
                         moe_stream_t stream) {
  MOE_TRY(validate_i8(rows, N, K));
  if ((!is_dtype(x_dtype) && x_dtype != MOE_I8) || !is_dtype(y_dtype)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(need(x, rows));
  if (x_dtype == MOE_I8) MOE_TRY(need(x_scale, rows, 4));
  else if (x_scale != nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(need(W, 1));
  MOE_TRY(need(w_scale, 1, 4));
  MOE_TRY(optional(bias, 4));
  MOE_TRY(need(y, rows));
  MOE_TRY(check_ws(ws, ws_bytes, kErrBytes + i8_linear_scratch(rows, N, K)));
  if (rows == 0) return MOE_OK;
  MOE_CUDA(launch_linear_i8(rows, N, K, x, x_dtype, x_scale, W, w_scale, bias, y, y_dtype,
                            past_error_word(ws), static_cast<int*>(ws), stream));
  return MOE_OK;
}

}  // extern "C"
