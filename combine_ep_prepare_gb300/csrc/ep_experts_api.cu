// ep_experts_api.cu -- the C ABI of the expert products and the router:
// host-side validation and parameters.  Like the row calls these only enqueue
// work on the stream: no allocation, no host synchronisation.
#include <cmath>

#include "ep_api_checks.h"

namespace {

using namespace ep::checks;
using ep::LayerInfo;

// Feature counts: rows of 16-byte vectors, bounded so that 32-bit column
// indices and the tile counts of EP_MAX_EXPERTS experts hold.
ep_status_t check_features(int64_t n, const char* name) {
  if (n < 8 || n % 8 != 0 || n > (1 << 20))
    return fail(EP_ERR_SHAPE, "%s %lld must be a positive multiple of 8, at most 2^20", name, (long long)n);
  return EP_OK;
}

ep_status_t layer(const ep_handle_t& h, const LayerInfo** L) { return ep::api_expert_layer(h, L); }

ep::ProductParams product_params(const LayerInfo* L, const ep_handle_t& h, int kind, int64_t N, int64_t K) {
  ep::ProductParams p;
  p.hdr = at<int>(h.mem, 0);
  p.counts = at<int>(h.mem, L->lay.counts);
  p.offsets = at<int>(h.mem, L->lay.offsets);
  p.E = own_experts(L);
  p.R = static_cast<int>(L->R);
  p.kind = kind;
  p.dtype = static_cast<int>(L->cfg.dtype);
  p.out_f32 = p.dtype == EP_DTYPE_FP32;
  p.accumulate = 0;
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.a = p.b = p.pre = nullptr;
  p.out = p.out2 = nullptr;
  return p;
}

ep_status_t enqueue(const ep::ProductParams& p, const char* where, void* stream) {
  int sms = 0;
  ep_status_t st = ep::api_device(&sms);
  if (st != EP_OK) return st;
  if (p.R == 0 && p.kind != ep::kProdWgrad) return EP_OK;
  const cudaError_t e = p.dtype == EP_DTYPE_FP32 ? ep::launch_product_simt(p, sms, static_cast<cudaStream_t>(stream))
                                                 : ep::launch_product_tc(p, sms, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(1);
  if (e != cudaSuccess) return ep::api_cuda_fail(e, where);
  return EP_OK;
}

ep_status_t w4(ep_handle_t h, bool gated, const void* x, const uint8_t* wq, const void* scales, int64_t N,
               int64_t K, int64_t group, void* out, const char* where, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = layer(h, &L);
  if (st != EP_OK) return st;
  if (L->cfg.dtype == EP_DTYPE_FP32)
    return fail(EP_ERR_INVALID_ARG, "%s takes bf16 and fp16 payloads", where);
  if ((st = check_features(N, "out_features")) != EP_OK) return st;
  if ((st = check_features(K, "in_features")) != EP_OK) return st;
  if (group != 32 && group != 64 && group != 128)
    return fail(EP_ERR_INVALID_ARG, "%s: group %lld is not 32, 64 or 128", where, (long long)group);
  if (K % group != 0) return fail(EP_ERR_SHAPE, "%s: in_features %lld is not a multiple of the group", where, (long long)K);
  if ((st = check_ptr(x, "x")) != EP_OK) return st;
  if ((st = check_ptr(wq, "wq")) != EP_OK) return st;
  if ((st = check_ptr(scales, "scales")) != EP_OK) return st;
  if ((st = check_ptr(out, "out")) != EP_OK) return st;
  int sms = 0;
  if ((st = ep::api_device(&sms)) != EP_OK) return st;
  ep::W4Params p;
  p.hdr = at<int>(h.mem, 0);
  p.counts = at<int>(h.mem, L->lay.counts);
  p.offsets = at<int>(h.mem, L->lay.offsets);
  p.E = own_experts(L);
  p.R = static_cast<int>(L->R);
  p.dtype = static_cast<int>(L->cfg.dtype);
  p.N = static_cast<int>(gated ? 2 * N : N);
  p.K = static_cast<int>(K);
  p.group = static_cast<int>(group);
  p.swiglu = gated;
  p.x = x;
  p.wq = wq;
  p.scales = scales;
  p.out = out;
  if (p.R == 0) return EP_OK;
  const cudaError_t e = ep::launch_w4(p, sms, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(1);
  if (e != cudaSuccess) return ep::api_cuda_fail(e, where);
  return EP_OK;
}

ep_status_t router_params(const ep_router_config_t& c, int64_t T, const void* logits, ep::RouterParams* p) {
  const ep_status_t st = router_config(c, T, p);
  if (st != EP_OK) return st;
  p->logits = logits;
  return T > 0 ? check_ptr(logits, "logits", c.dtype == EP_DTYPE_FP32 ? 4 : 2) : EP_OK;
}

}  // namespace

namespace ep {
namespace checks {

ep_status_t router_config(const ep_router_config_t& c, int64_t T, RouterParams* p) {
  if (c.num_experts < 1 || c.num_experts > EP_MAX_EXPERTS)
    return fail(EP_ERR_LIMIT, "%s %lld outside [1, EP_MAX_EXPERTS]", "num_experts", (long long)c.num_experts);
  if (c.top_k < 1 || c.top_k > EP_MAX_TOPK || c.top_k > c.num_experts)
    return fail(EP_ERR_LIMIT, "%s %lld outside [1, min(EP_MAX_TOPK, num_experts)]", "top_k", (long long)c.top_k);
  if (c.num_groups < 1 || c.num_groups > 32 || c.num_experts % c.num_groups != 0)
    return fail(EP_ERR_LIMIT, "%s %lld must lie in [1, 32] and divide num_experts", "num_groups", (long long)c.num_groups);
  if (c.topk_groups < 1 || c.topk_groups > c.num_groups)
    return fail(EP_ERR_INVALID_ARG, "%s %lld outside [1, num_groups]", "topk_groups", (long long)c.topk_groups);
  if (c.score != EP_SCORE_SOFTMAX && c.score != EP_SCORE_SIGMOID)
    return fail(EP_ERR_INVALID_ARG, "%s %lld is not an ep_score_t", "score", (long long)c.score);
  if (c.normalize != 0 && c.normalize != 1)
    return fail(EP_ERR_INVALID_ARG, "%s %lld must be 0 or 1", "normalize", (long long)c.normalize);
  if (c.dtype != EP_DTYPE_BF16 && c.dtype != EP_DTYPE_FP16 && c.dtype != EP_DTYPE_FP32)
    return fail(EP_ERR_INVALID_ARG, "%s %lld is not an ep_dtype_t", "dtype", (long long)c.dtype);
  if (!std::isfinite(c.scale)) return fail(EP_ERR_INVALID_ARG, "%s is not finite", "scale");
  if (T < 0 || T > (1LL << 24) / c.top_k)
    return fail(EP_ERR_SHAPE, "%s %lld: num_tokens*top_k must lie in [0, 2^24]", "num_tokens", (long long)T);
  p->T = static_cast<int>(T);
  p->E = static_cast<int>(c.num_experts);
  p->K = static_cast<int>(c.top_k);
  p->groups = static_cast<int>(c.num_groups);
  p->kept = static_cast<int>(c.topk_groups);
  p->sigmoid = c.score == EP_SCORE_SIGMOID;
  p->normalize = static_cast<int>(c.normalize);
  p->dtype = static_cast<int>(c.dtype);
  p->scale = c.scale;
  p->logits = nullptr;
  p->bias = nullptr;
  p->idx = nullptr;
  p->w = nullptr;
  p->grad = nullptr;
  p->grad_logits = nullptr;
  return EP_OK;
}

}  // namespace checks
}  // namespace ep

extern "C" {

ep_status_t ep_expert_gemm(ep_handle_t h, const void* x, const void* w, int64_t out_features,
                           int64_t in_features, void* y, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = layer(h, &L);
  if (st != EP_OK) return st;
  if ((st = check_features(out_features, "out_features")) != EP_OK) return st;
  if ((st = check_features(in_features, "in_features")) != EP_OK) return st;
  if ((st = check_ptr(x, "x")) != EP_OK) return st;
  if ((st = check_ptr(w, "w")) != EP_OK) return st;
  if ((st = check_ptr(y, "y")) != EP_OK) return st;
  ep::ProductParams p = product_params(L, h, ep::kProdFwd, out_features, in_features);
  p.a = x;
  p.b = w;
  p.out = y;
  return enqueue(p, "ep_expert_gemm launch", stream);
}

ep_status_t ep_expert_gemm_swiglu(ep_handle_t h, const void* x, const void* w, int64_t ffn_features,
                                  int64_t in_features, void* pre, void* act, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = layer(h, &L);
  if (st != EP_OK) return st;
  if ((st = check_features(ffn_features, "ffn_features")) != EP_OK) return st;
  if ((st = check_features(in_features, "in_features")) != EP_OK) return st;
  if ((st = check_ptr(x, "x")) != EP_OK) return st;
  if ((st = check_ptr(w, "w")) != EP_OK) return st;
  if (pre != nullptr && (st = check_ptr(pre, "pre")) != EP_OK) return st;
  if ((st = check_ptr(act, "act")) != EP_OK) return st;
  ep::ProductParams p = product_params(L, h, ep::kProdFwdSwiglu, 2 * ffn_features, in_features);
  p.a = x;
  p.b = w;
  p.out = act;
  p.out2 = pre;
  return enqueue(p, "ep_expert_gemm_swiglu launch", stream);
}

ep_status_t ep_expert_dgrad(ep_handle_t h, const void* dy, const void* w, int64_t out_features,
                            int64_t in_features, void* dx, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = layer(h, &L);
  if (st != EP_OK) return st;
  if ((st = check_features(out_features, "out_features")) != EP_OK) return st;
  if ((st = check_features(in_features, "in_features")) != EP_OK) return st;
  if ((st = check_ptr(dy, "dy")) != EP_OK) return st;
  if ((st = check_ptr(w, "w")) != EP_OK) return st;
  if ((st = check_ptr(dx, "dx")) != EP_OK) return st;
  ep::ProductParams p = product_params(L, h, ep::kProdDgrad, out_features, in_features);
  p.a = dy;
  p.b = w;
  p.out = dx;
  return enqueue(p, "ep_expert_dgrad launch", stream);
}

ep_status_t ep_expert_dgrad_swiglu(ep_handle_t h, const void* dy, const void* w, const void* pre,
                                   int64_t out_features, int64_t ffn_features, void* dpre, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = layer(h, &L);
  if (st != EP_OK) return st;
  if ((st = check_features(out_features, "out_features")) != EP_OK) return st;
  if ((st = check_features(ffn_features, "ffn_features")) != EP_OK) return st;
  if ((st = check_ptr(dy, "dy")) != EP_OK) return st;
  if ((st = check_ptr(w, "w")) != EP_OK) return st;
  if ((st = check_ptr(pre, "pre")) != EP_OK) return st;
  if ((st = check_ptr(dpre, "dpre")) != EP_OK) return st;
  ep::ProductParams p = product_params(L, h, ep::kProdDgradSwiglu, out_features, ffn_features);
  p.a = dy;
  p.b = w;
  p.pre = pre;
  p.out = dpre;
  return enqueue(p, "ep_expert_dgrad_swiglu launch", stream);
}

ep_status_t ep_expert_wgrad(ep_handle_t h, const void* dy, const void* x, int64_t out_features,
                            int64_t in_features, void* dw, int64_t dw_dtype, int accumulate, void* stream) {
  const LayerInfo* L = nullptr;
  ep_status_t st = layer(h, &L);
  if (st != EP_OK) return st;
  if ((st = check_features(out_features, "out_features")) != EP_OK) return st;
  if ((st = check_features(in_features, "in_features")) != EP_OK) return st;
  if (dw_dtype != L->cfg.dtype && dw_dtype != EP_DTYPE_FP32)
    return fail(EP_ERR_INVALID_ARG, "%s %lld is neither the layer's payload type nor fp32", "dw_dtype", (long long)dw_dtype);
  if (accumulate != 0 && accumulate != 1)
    return fail(EP_ERR_INVALID_ARG, "%s %lld must be 0 or 1", "accumulate", accumulate);
  if ((st = check_ptr(dy, "dy")) != EP_OK) return st;
  if ((st = check_ptr(x, "x")) != EP_OK) return st;
  if ((st = check_ptr(dw, "dw")) != EP_OK) return st;
  ep::ProductParams p = product_params(L, h, ep::kProdWgrad, out_features, in_features);
  p.a = dy;
  p.b = x;
  p.out = dw;
  p.out_f32 = dw_dtype == EP_DTYPE_FP32;
  p.accumulate = accumulate;
  return enqueue(p, "ep_expert_wgrad launch", stream);
}

ep_status_t ep_expert_gemv_w4(ep_handle_t h, const void* x, const uint8_t* wq, const void* scales,
                              int64_t out_features, int64_t in_features, int64_t group, void* y, void* stream) {
  return w4(h, false, x, wq, scales, out_features, in_features, group, y, "ep_expert_gemv_w4", stream);
}

ep_status_t ep_expert_gemv_w4_swiglu(ep_handle_t h, const void* x, const uint8_t* wq, const void* scales,
                                     int64_t ffn_features, int64_t in_features, int64_t group, void* act,
                                     void* stream) {
  return w4(h, true, x, wq, scales, ffn_features, in_features, group, act, "ep_expert_gemv_w4_swiglu", stream);
}

ep_status_t ep_router(ep_router_config_t config, const void* logits, const float* bias, int64_t num_tokens,
                      int64_t* topk_idx, float* topk_weights, void* stream) {
  ep::RouterParams p;
  ep_status_t st = router_params(config, num_tokens, logits, &p);
  if (st != EP_OK) return st;
  if (bias != nullptr) {
    if (!p.sigmoid) return fail(EP_ERR_INVALID_ARG, "%s: a selection bias needs the sigmoid score", "bias");
    if ((st = check_ptr(bias, "bias", 4)) != EP_OK) return st;
  }
  if (num_tokens > 0) {
    if ((st = check_ptr(topk_idx, "topk_idx", 8)) != EP_OK) return st;
    if ((st = check_ptr(topk_weights, "topk_weights", 4)) != EP_OK) return st;
  }
  int sms = 0;
  if ((st = ep::api_device(&sms)) != EP_OK) return st;
  if (num_tokens == 0) return EP_OK;
  p.bias = bias;
  p.idx = reinterpret_cast<long long*>(topk_idx);
  p.w = topk_weights;
  const cudaError_t e = ep::launch_router(p, sms, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(1);
  if (e != cudaSuccess) return ep::api_cuda_fail(e, "ep_router launch");
  return EP_OK;
}

ep_status_t ep_router_bwd(ep_router_config_t config, const void* logits, const int64_t* topk_idx,
                          const float* grad_topk_weights, int64_t num_tokens, void* grad_logits, void* stream) {
  ep::RouterParams p;
  ep_status_t st = router_params(config, num_tokens, logits, &p);
  if (st != EP_OK) return st;
  if (num_tokens > 0) {
    if ((st = check_ptr(topk_idx, "topk_idx", 8)) != EP_OK) return st;
    if ((st = check_ptr(grad_topk_weights, "grad_topk_weights", 4)) != EP_OK) return st;
    if ((st = check_ptr(grad_logits, "grad_logits", p.dtype == EP_DTYPE_FP32 ? 4 : 2)) != EP_OK) return st;
  }
  int sms = 0;
  if ((st = ep::api_device(&sms)) != EP_OK) return st;
  if (num_tokens == 0) return EP_OK;
  p.idx = const_cast<long long*>(reinterpret_cast<const long long*>(topk_idx));
  p.grad = grad_topk_weights;
  p.grad_logits = grad_logits;
  const cudaError_t e = ep::launch_router_bwd(p, sms, static_cast<cudaStream_t>(stream));
  ep::api_count_launches(1);
  if (e != cudaSuccess) return ep::api_cuda_fail(e, "ep_router_bwd launch");
  return EP_OK;
}

}  // extern "C"
