// ep_f8_api.cu -- the C ABI of the norm, the 8-bit rows and products, and a few
// tokens' whole layer: host-side validation and parameters.  Like the other
// calls these only enqueue work on the stream.
#include <cmath>

#include "ep_api_checks.h"
#include "ep_f8.cuh"
#include "ep_moe_few.cuh"

namespace {

using namespace ep::checks;
using ep::LayerInfo;

bool known_dtype(int64_t d) { return d == EP_DTYPE_BF16 || d == EP_DTYPE_FP16 || d == EP_DTYPE_FP32; }

// Rows of the row calls: whole 16-byte vectors held on chip.
ep_status_t check_rows(int64_t rows, int64_t n, int64_t most, int64_t dtype, bool f8, const char* name) {
  if (!known_dtype(dtype)) return fail(EP_ERR_INVALID_ARG, "%s %lld is not an ep_dtype_t", "dtype", (long long)dtype);
  if (rows < 0 || rows > 0x7fffffffLL) return fail(EP_ERR_SHAPE, "%s %lld outside [0, 2^31)", name, (long long)rows);
  if (n < 8 || n % (f8 ? 16 : 8) != 0)
    return fail(EP_ERR_SHAPE, f8 ? "%s %lld must be a positive multiple of 16" : "%s %lld must be a positive multiple of 8",
                "the row length", (long long)n);
  if (n > most) return fail(EP_ERR_LIMIT, "%s %lld is too long", "the row length", (long long)n);
  return EP_OK;
}

ep_status_t check_f8_features(int64_t n, const char* name, bool gated = false) {
  if (n < 16 || n % 16 != 0 || n > (1 << 20))
    return fail(EP_ERR_SHAPE, "%s %lld must be a positive multiple of 16, at most 2^20", name, (long long)n);
  if (gated && n % ep::kF8Block != 0)
    return fail(EP_ERR_SHAPE, "%s %lld must be a multiple of 128: gate and up rows have scale blocks of their own", name, (long long)n);
  return EP_OK;
}

ep_status_t f8_layer(const ep_handle_t& h, const LayerInfo** L, const char* where) {
  const ep_status_t st = ep::api_expert_layer(h, L);
  if (st != EP_OK) return st;
  if ((*L)->cfg.dtype == EP_DTYPE_FP32) return fail(EP_ERR_INVALID_ARG, "%s takes bf16 and fp16 payloads", where);
  return EP_OK;
}

// Rows, their scales, the weights and theirs.
ep_status_t check_operands(const void* a, const float* as, const void* w, const float* ws, const char* a_name, const char* as_name) {
  ep_status_t st;
  if ((st = check_ptr(a, a_name)) != EP_OK) return st;
  if ((st = check_ptr(as, as_name)) != EP_OK) return st;
  if ((st = check_ptr(w, "w")) != EP_OK) return st;
  return check_ptr(ws, "w_scales", 4);
}

ep::F8Params f8_params(const LayerInfo* L, const ep_handle_t& h, int kind, const uint8_t* a, const float* as,
                       const uint8_t* w, const float* ws, int64_t N, int64_t K) {
  ep::F8Params p = {};
  p.hdr = at<int>(h.mem, 0);
  p.counts = at<int>(h.mem, L->lay.counts);
  p.offsets = at<int>(h.mem, L->lay.offsets);
  p.E = own_experts(L);
  p.R = static_cast<int>(L->R);
  p.kind = kind;
  p.dtype = static_cast<int>(L->cfg.dtype);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.a = a;
  p.as = as;
  p.w = w;
  p.ws = ws;
  return p;
}

ep_status_t enqueue(const ep::F8Params& p, const char* where, void* stream) {
  int sms = 0;
  const ep_status_t st = ep::api_device(&sms);
  if (st != EP_OK) return st;
  if (p.R == 0) return EP_OK;
  const cudaError_t e = ep::launch_product_f8(p, sms, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(1);
  return e == cudaSuccess ? EP_OK : ep::api_cuda_fail(e, where);
}

ep_status_t few_config(const ep_moe_few_config_t& c, int64_t T, ep::RouterParams* r) {
  const ep_status_t st = router_config(c.router, 0, r);
  if (st != EP_OK) return st;
  if (T < 0 || T > EP_MAX_FEW_TOKENS) return fail(EP_ERR_SHAPE, "%s %lld outside [0, EP_MAX_FEW_TOKENS]", "num_tokens", (long long)T);
  r->T = static_cast<int>(T);
  if (c.dtype != EP_DTYPE_BF16 && c.dtype != EP_DTYPE_FP16)
    return fail(EP_ERR_INVALID_ARG, "%s %lld: ep_moe_few takes bf16 and fp16", "dtype", (long long)c.dtype);
  if (c.weight_f8 != 0 && c.weight_f8 != 1) return fail(EP_ERR_INVALID_ARG, "%s %lld must be 0 or 1", "weight_f8", (long long)c.weight_f8);
  const int64_t h = c.weight_f8 ? 16 : 8, f = c.weight_f8 ? ep::kF8Block : 8;
  if (c.hidden < h || c.hidden % h != 0 || c.hidden > EP_MAX_NORM_HIDDEN)
    return fail(EP_ERR_SHAPE, "%s %lld must be a positive multiple of 8 (8-bit weights: 16), at most 32768", "hidden", (long long)c.hidden);
  if (c.ffn < f || c.ffn % f != 0 || c.ffn > EP_MAX_NORM_HIDDEN)
    return fail(EP_ERR_SHAPE, "%s %lld must be a positive multiple of 8 (8-bit weights: 128), at most 32768", "ffn", (long long)c.ffn);
  return EP_OK;
}

}  // namespace

extern "C" {

ep_status_t ep_rmsnorm(const void* x, const void* residual, const void* weight, int64_t num_tokens, int64_t hidden,
                       int64_t dtype, float eps, void* sum, void* y, uint8_t* q, float* scales, void* stream) {
  ep_status_t st = check_rows(num_tokens, hidden, EP_MAX_NORM_HIDDEN, dtype, q != nullptr, "num_tokens");
  if (st != EP_OK) return st;
  if (!std::isfinite(eps) || eps < 0.0f) return fail(EP_ERR_INVALID_ARG, "%s is negative or not finite", "eps");
  if (num_tokens > 0) {  // no tokens: buffers of no bytes may have any address
    if ((q == nullptr) != (scales == nullptr)) return fail(EP_ERR_INVALID_ARG, "%s go together", "q and scales");
    if (sum != nullptr && residual == nullptr) return fail(EP_ERR_INVALID_ARG, "%s needs a residual", "sum");
    if (sum == nullptr && y == nullptr && q == nullptr) return fail(EP_ERR_INVALID_ARG, "%s are all NULL", "sum, y and q");
    if ((st = check_ptr(x, "x")) != EP_OK) return st;
    if ((st = check_ptr(weight, "weight")) != EP_OK) return st;
    if (residual != nullptr && (st = check_ptr(residual, "residual")) != EP_OK) return st;
    if (sum != nullptr && (st = check_ptr(sum, "sum")) != EP_OK) return st;
    if (y != nullptr && (st = check_ptr(y, "y")) != EP_OK) return st;
    if (q != nullptr && (st = check_ptr(q, "q")) != EP_OK) return st;
    if (scales != nullptr && (st = check_ptr(scales, "scales")) != EP_OK) return st;
  }
  int sms = 0;
  if ((st = ep::api_device(&sms)) != EP_OK) return st;
  if (num_tokens == 0) return EP_OK;
  ep::NormParams p = {};
  p.T = static_cast<int>(num_tokens);
  p.H = static_cast<int>(hidden);
  p.dtype = static_cast<int>(dtype);
  p.eps = eps;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.sum = sum;
  p.y = y;
  p.q = q;
  p.scales = scales;
  const cudaError_t e = ep::launch_norm(p, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(1);
  return e == cudaSuccess ? EP_OK : ep::api_cuda_fail(e, "ep_rmsnorm launch");
}

ep_status_t ep_rmsnorm_bwd_workspace(int64_t num_tokens, int64_t hidden, size_t* bytes) {
  if (bytes == nullptr) return fail(EP_ERR_INVALID_ARG, "%s is NULL", "bytes");
  const ep_status_t st = check_rows(num_tokens, hidden, EP_MAX_NORM_HIDDEN, EP_DTYPE_FP32, false, "num_tokens");
  if (st != EP_OK) return st;
  *bytes = sizeof(float) * static_cast<size_t>(hidden) * static_cast<size_t>(ep::norm_bwd_parts(num_tokens, hidden));
  return EP_OK;
}

ep_status_t ep_rmsnorm_bwd(const void* grad_y, const void* h, const void* weight, const void* grad_sum,
                           int64_t num_tokens, int64_t hidden, int64_t dtype, float eps, void* grad_h,
                           float* grad_weight, int accumulate, void* workspace, void* stream) {
  ep_status_t st = check_rows(num_tokens, hidden, EP_MAX_NORM_HIDDEN, dtype, false, "num_tokens");
  if (st != EP_OK) return st;
  if (!std::isfinite(eps) || eps < 0.0f) return fail(EP_ERR_INVALID_ARG, "%s is negative or not finite", "eps");
  if (accumulate != 0 && accumulate != 1) return fail(EP_ERR_INVALID_ARG, "%s %lld must be 0 or 1", "accumulate", accumulate);
  if ((st = check_ptr(grad_weight, "grad_weight")) != EP_OK) return st;
  if (num_tokens > 0) {
    if ((st = check_ptr(grad_y, "grad_y")) != EP_OK) return st;
    if ((st = check_ptr(h, "h")) != EP_OK) return st;
    if ((st = check_ptr(weight, "weight")) != EP_OK) return st;
    if (grad_sum != nullptr && (st = check_ptr(grad_sum, "grad_sum")) != EP_OK) return st;
    if ((st = check_ptr(grad_h, "grad_h")) != EP_OK) return st;
    if ((st = check_ptr(workspace, "workspace")) != EP_OK) return st;
  }
  int sms = 0;
  if ((st = ep::api_device(&sms)) != EP_OK) return st;
  ep::NormParams p = {};
  p.T = static_cast<int>(num_tokens);
  p.H = static_cast<int>(hidden);
  p.dtype = static_cast<int>(dtype);
  p.eps = eps;
  p.x = h;
  p.weight = weight;
  p.dy = grad_y;
  p.dsum = grad_sum;
  p.dh = grad_h;
  p.dw = grad_weight;
  p.accumulate = accumulate;
  p.partial = static_cast<float*>(workspace);
  const cudaError_t e = ep::launch_norm_bwd(p, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(num_tokens > 0 ? 2 : 1);
  return e == cudaSuccess ? EP_OK : ep::api_cuda_fail(e, "ep_rmsnorm_bwd launch");
}

ep_status_t ep_quantize_rows(const void* x, int64_t rows, int64_t features, int64_t dtype, uint8_t* q, float* scales,
                             void* stream) {
  ep_status_t st = check_rows(rows, features, 1 << 20, dtype, true, "rows");
  if (st != EP_OK) return st;
  if (rows > 0) {
    if ((st = check_ptr(x, "x")) != EP_OK) return st;
    if ((st = check_ptr(q, "q")) != EP_OK) return st;
    if ((st = check_ptr(scales, "scales")) != EP_OK) return st;
  }
  int sms = 0;
  if ((st = ep::api_device(&sms)) != EP_OK) return st;
  if (rows == 0) return EP_OK;
  ep::QuantParams p = {};
  p.R = static_cast<int>(rows);
  p.n = static_cast<int>(features);
  p.dtype = static_cast<int>(dtype);
  p.x = x;
  p.q = q;
  p.scales = scales;
  const cudaError_t e = ep::launch_quantize(p, sms, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(1);
  return e == cudaSuccess ? EP_OK : ep::api_cuda_fail(e, "ep_quantize_rows launch");
}

ep_status_t ep_expert_quantize(ep_handle_t h, const void* x, int64_t features, uint8_t* q, float* scales, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = f8_layer(h, &L, "ep_expert_quantize");
  if (st != EP_OK) return st;
  if ((st = check_f8_features(features, "features")) != EP_OK) return st;
  if ((st = check_ptr(x, "x")) != EP_OK) return st;
  if ((st = check_ptr(q, "q")) != EP_OK) return st;
  if ((st = check_ptr(scales, "scales")) != EP_OK) return st;
  int sms = 0;
  if ((st = ep::api_device(&sms)) != EP_OK) return st;
  if (L->R == 0) return EP_OK;
  ep::QuantParams p = {};
  p.hdr = at<int>(h.mem, 0);
  p.counts = at<int>(h.mem, L->lay.counts);
  p.offsets = at<int>(h.mem, L->lay.offsets);
  p.E = own_experts(L);
  p.R = static_cast<int>(L->R);
  p.n = static_cast<int>(features);
  p.dtype = static_cast<int>(L->cfg.dtype);
  p.x = x;
  p.q = q;
  p.scales = scales;
  const cudaError_t e = ep::launch_quantize(p, sms, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(1);
  return e == cudaSuccess ? EP_OK : ep::api_cuda_fail(e, "ep_expert_quantize launch");
}

ep_status_t ep_expert_gemm_f8(ep_handle_t h, const uint8_t* x, const float* x_scales, const uint8_t* w,
                              const float* w_scales, int64_t out_features, int64_t in_features, void* y, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = f8_layer(h, &L, "ep_expert_gemm_f8");
  if (st != EP_OK) return st;
  if ((st = check_f8_features(out_features, "out_features")) != EP_OK) return st;
  if ((st = check_f8_features(in_features, "in_features")) != EP_OK) return st;
  if ((st = check_operands(x, x_scales, w, w_scales, "x", "x_scales")) != EP_OK) return st;
  if ((st = check_ptr(y, "y")) != EP_OK) return st;
  ep::F8Params p = f8_params(L, h, ep::kProdFwd, x, x_scales, w, w_scales, out_features, in_features);
  p.out = y;
  return enqueue(p, "ep_expert_gemm_f8 launch", stream);
}

ep_status_t ep_expert_gemm_f8_swiglu(ep_handle_t h, const uint8_t* x, const float* x_scales, const uint8_t* w,
                                     const float* w_scales, int64_t ffn_features, int64_t in_features, void* pre,
                                     void* act, uint8_t* act_q, float* act_scales, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = f8_layer(h, &L, "ep_expert_gemm_f8_swiglu");
  if (st != EP_OK) return st;
  if ((st = check_f8_features(ffn_features, "ffn_features", true)) != EP_OK) return st;
  if ((st = check_f8_features(in_features, "in_features")) != EP_OK) return st;
  if ((st = check_operands(x, x_scales, w, w_scales, "x", "x_scales")) != EP_OK) return st;
  if ((act_q == nullptr) != (act_scales == nullptr)) return fail(EP_ERR_INVALID_ARG, "%s go together", "act_q and act_scales");
  if (pre == nullptr && act == nullptr && act_q == nullptr) return fail(EP_ERR_INVALID_ARG, "%s are all NULL", "pre, act and act_q");
  if (pre != nullptr && (st = check_ptr(pre, "pre")) != EP_OK) return st;
  if (act != nullptr && (st = check_ptr(act, "act")) != EP_OK) return st;
  if (act_q != nullptr && (st = check_ptr(act_q, "act_q")) != EP_OK) return st;
  if (act_scales != nullptr && (st = check_ptr(act_scales, "act_scales")) != EP_OK) return st;
  ep::F8Params p = f8_params(L, h, ep::kProdFwdSwiglu, x, x_scales, w, w_scales, 2 * ffn_features, in_features);
  p.out = act;
  p.pre = pre;
  p.q = act_q;
  p.qs = act_scales;
  return enqueue(p, "ep_expert_gemm_f8_swiglu launch", stream);
}

ep_status_t ep_expert_dgrad_f8(ep_handle_t h, const uint8_t* dy, const float* dy_scales, const uint8_t* w,
                               const float* w_scales, int64_t out_features, int64_t in_features, void* dx, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = f8_layer(h, &L, "ep_expert_dgrad_f8");
  if (st != EP_OK) return st;
  if ((st = check_f8_features(out_features, "out_features")) != EP_OK) return st;
  if ((st = check_f8_features(in_features, "in_features")) != EP_OK) return st;
  if ((st = check_operands(dy, dy_scales, w, w_scales, "dy", "dy_scales")) != EP_OK) return st;
  if ((st = check_ptr(dx, "dx")) != EP_OK) return st;
  ep::F8Params p = f8_params(L, h, ep::kProdDgrad, dy, dy_scales, w, w_scales, out_features, in_features);
  p.out = dx;
  return enqueue(p, "ep_expert_dgrad_f8 launch", stream);
}

ep_status_t ep_expert_dgrad_f8_swiglu(ep_handle_t h, const uint8_t* dy, const float* dy_scales, const uint8_t* w,
                                      const float* w_scales, const void* pre, int64_t out_features,
                                      int64_t ffn_features, void* dpre, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = f8_layer(h, &L, "ep_expert_dgrad_f8_swiglu");
  if (st != EP_OK) return st;
  if ((st = check_f8_features(out_features, "out_features")) != EP_OK) return st;
  if ((st = check_f8_features(ffn_features, "ffn_features", true)) != EP_OK) return st;
  if ((st = check_operands(dy, dy_scales, w, w_scales, "dy", "dy_scales")) != EP_OK) return st;
  if ((st = check_ptr(pre, "pre")) != EP_OK) return st;
  if ((st = check_ptr(dpre, "dpre")) != EP_OK) return st;
  ep::F8Params p = f8_params(L, h, ep::kProdDgradSwiglu, dy, dy_scales, w, w_scales, out_features, ffn_features);
  p.pre_in = pre;
  p.out = dpre;
  return enqueue(p, "ep_expert_dgrad_f8_swiglu launch", stream);
}

ep_status_t ep_moe_few_workspace(ep_moe_few_config_t config, int64_t num_tokens, size_t* bytes) {
  if (bytes == nullptr) return fail(EP_ERR_INVALID_ARG, "%s is NULL", "bytes");
  ep::RouterParams r;
  const ep_status_t st = few_config(config, num_tokens, &r);
  if (st != EP_OK) return st;
  *bytes = ep::few_layout(num_tokens, r.E, r.K, config.hidden, config.ffn, config.weight_f8 != 0).total;
  return EP_OK;
}

ep_status_t ep_moe_few(ep_moe_few_config_t config, const void* x, const void* gate, const float* bias, const void* w13,
                       const float* w13_scales, const void* w2, const float* w2_scales, int64_t num_tokens, void* out,
                       int64_t* topk_idx, float* topk_weights, void* workspace, void* stream) {
  ep::FewParams p = {};
  ep_status_t st = few_config(config, num_tokens, &p.router);
  if (st != EP_OK) return st;
  const bool f8 = config.weight_f8 != 0;
  if (!f8 && (w13_scales != nullptr || w2_scales != nullptr))
    return fail(EP_ERR_INVALID_ARG, "%s belong to 8-bit weights", "w13_scales and w2_scales");
  if (bias != nullptr) {
    if (!p.router.sigmoid) return fail(EP_ERR_INVALID_ARG, "%s: a selection bias needs the sigmoid score", "bias");
    if ((st = check_ptr(bias, "bias", 4)) != EP_OK) return st;
  }
  if (num_tokens > 0) {
    if ((st = check_ptr(x, "x")) != EP_OK) return st;
    if ((st = check_ptr(gate, "gate")) != EP_OK) return st;
    if ((st = check_ptr(w13, "w13")) != EP_OK) return st;
    if ((st = check_ptr(w2, "w2")) != EP_OK) return st;
    if (f8 && (st = check_ptr(w13_scales, "w13_scales", 4)) != EP_OK) return st;
    if (f8 && (st = check_ptr(w2_scales, "w2_scales", 4)) != EP_OK) return st;
    if ((st = check_ptr(out, "out")) != EP_OK) return st;
    if ((st = check_ptr(topk_idx, "topk_idx", 8)) != EP_OK) return st;
    if ((st = check_ptr(topk_weights, "topk_weights", 4)) != EP_OK) return st;
    if ((st = check_ptr(workspace, "workspace", 256)) != EP_OK) return st;
  }
  int sms = 0;
  if ((st = ep::api_device(&sms)) != EP_OK) return st;
  if (num_tokens == 0) return EP_OK;
  p.T = static_cast<int>(num_tokens);
  p.E = p.router.E;
  p.K = p.router.K;
  p.H = static_cast<int>(config.hidden);
  p.F = static_cast<int>(config.ffn);
  p.dtype = static_cast<int>(config.dtype);
  p.gate_dtype = p.router.dtype;
  p.f8 = f8;
  p.x = x;
  p.gate = gate;
  p.w13 = w13;
  p.s13 = w13_scales;
  p.w2 = w2;
  p.s2 = w2_scales;
  p.out = out;
  p.idx = reinterpret_cast<long long*>(topk_idx);
  p.w = topk_weights;
  const ep::FewLayout l = ep::few_layout(p.T, p.E, p.K, p.H, p.F, f8);
  p.hdr = at<int>(workspace, 0);
  p.done = at<int>(workspace, l.done);
  p.written = at<int>(workspace, l.written);
  p.zeros = l.zeros;
  p.logits = at<float>(workspace, l.logits);
  p.act = at<char>(workspace, l.act);
  p.xq = at<__half>(workspace, l.xq);
  p.xs = at<float>(workspace, l.xs);
  p.aq = at<__half>(workspace, l.aq);
  p.as = at<float>(workspace, l.as);
  p.part = at<float>(workspace, l.part);
  p.router.logits = p.logits;
  p.router.dtype = EP_DTYPE_FP32;
  p.router.bias = bias;
  const cudaError_t e = ep::launch_moe_few(p, sms, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(2);
  return e == cudaSuccess ? EP_OK : ep::api_cuda_fail(e, "ep_moe_few launch");
}

}  // extern "C"
