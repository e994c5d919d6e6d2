// ep_router.cu -- the router in front of prepare, and its gradient.
//
// Per token with logits z[0..E): selection values v_e = z_e (softmax) or
// sigmoid(z_e) + bias_e (sigmoid).  With groups, a group's rank is the sum of
// its two largest v and only the `kept` best groups' experts stay.  The K
// largest v are chosen in descending order, ties to the lowest index.  A
// logit or value that is -inf or NaN is never chosen; where fewer than K
// are left, the remaining ids are -1 and their weights 0.
//
// One warp per token: lane l holds the values of J experts from l J on as
// order-preserving unsigned keys (0 = cannot be chosen).  A round of the
// selection is one redux.sync maximum over the lanes' best keys; the lowest
// lane that holds it has the lowest index, since lanes hold runs of experts.
// Instruction issue bounds the kernel as it is (72% of the slots, 1,070 warp
// instructions a token, most of them the rounds and the exact sigmoids):
// 16,384 tokens x 256 experts, 8 groups, 8 choices take 20 us where
// the bytes alone would take 2.7.
#include "ep_router.cuh"

namespace ep {
namespace {

using namespace route;

constexpr int kWarps = 4;  // one for each of an SM's schedulers

template <typename T, int J>
__global__ void __launch_bounds__(kWarps * 32) ep_router_kernel(const RouterParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  int mine;
  float w;
  route_token<T, J>(p, t, lane, &mine, &w);
  if (lane < p.K) {
    p.idx[static_cast<long long>(t) * p.K + lane] = mine;
    p.w[static_cast<long long>(t) * p.K + lane] = w;
  }
}

// d loss / d logits, the choice held fixed.  With s_k the chosen scores, S
// their sum, w_k = s_k / S the normalised ones and g the gradient of the
// weights (times `scale`):
//   sigmoid              dz_k = s_k (1 - s_k) g_k
//   sigmoid, normalised  dz_k = w_k (1 - s_k) (g_k - sum g w)
//   softmax, normalised  dz_k = w_k (g_k - sum g w)
//   softmax              dz_e = p_e ([e chosen] g_e - sum_k g_k p_k), every e
// 1 - s is the sigmoid of -z: the difference would lose its digits from z = 8
// on and be 0 from 17 on.  Dividing s by S before anything else keeps the
// quotients of very small scores in range.
// The row is written once densely and the K chosen entries after it: bound by
// the write of [T][E].
template <typename T, int J>
__global__ void __launch_bounds__(kWarps * 32) ep_router_bwd_kernel(const RouterParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const long long row = static_cast<long long>(t) * p.E, krow = static_cast<long long>(t) * p.K;
  T* out = static_cast<T*>(p.grad_logits) + row;
  long long e = lane < p.K ? p.idx[krow + lane] : -1;
  if (e < 0 || e >= p.E) e = -1;
  const float g = e >= 0 ? p.grad[krow + lane] * p.scale : 0.0f;
  const float ze = e >= 0 ? logit<T>(p.logits, row + e) : -INFINITY;
  float d;
  if (p.sigmoid || p.normalize) {
    if (p.sigmoid) {
      float w = e >= 0 ? sigmoidf(ze) : 0.0f, inner = 0.0f;
      if (p.normalize) {
        const float S = warp_sum(w);
        w = S > 0.0f ? w / S : 0.0f;
        inner = warp_sum(g * w);
      }
      d = w * sigmoidf(-ze) * (g - inner);
    } else {
      const unsigned m = __reduce_max_sync(kAll, key_of(ze));
      const float x = exp_or_0(ze, m ? value_of(m) : 0.0f);
      const float S = warp_sum(x);
      const float w = S != 0.0f ? x / S : 0.0f;
      d = w * (g - warp_sum(g * w));
    }
    constexpr int kVec = 16 / sizeof(T);
    if (p.E % kVec == 0 && reinterpret_cast<uintptr_t>(p.grad_logits) % 16 == 0) {
      for (int i = lane * kVec; i < p.E; i += 32 * kVec) *reinterpret_cast<uint4*>(out + i) = make_uint4(0, 0, 0, 0);
    } else {
      for (int i = lane; i < p.E; i += 32) out[i] = from_f32<T>(0.0f);
    }
  } else {
    float z[J];
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      z[j] = lane + 32 * j < p.E ? logit<T>(p.logits, row + lane + 32 * j) : -INFINITY;
      m = max(m, key_of(z[j]));
    }
    m = __reduce_max_sync(kAll, m);
    const float zmax = m ? value_of(m) : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      z[j] = exp_or_0(z[j], zmax);
      s += z[j];
    }
    s = warp_sum(s);
    const float inv = s != 0.0f ? 1.0f / s : 0.0f;
    const float pe = exp_or_0(ze, zmax) * inv;
    const float inner = warp_sum(g * pe);
    d = pe * (g - inner);
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane + 32 * j < p.E) out[lane + 32 * j] = from_f32<T>(z[j] * inv * -inner);
  }
  __syncwarp();  // orders the dense writes before the chosen entries'
  if (e >= 0) out[e] = from_f32<T>(d);
}

template <typename T, bool bwd>
cudaError_t launch_typed(const RouterParams& p, cudaStream_t s) {
  const dim3 grid((p.T + kWarps - 1) / kWarps), block(kWarps * 32);
  const int j = (p.E + 31) / 32;
#define EP_ROUTER(JJ)                                                                   \
  if (j <= JJ) {                                                                        \
    if constexpr (bwd) return launch_pdl(ep_router_bwd_kernel<T, JJ>, grid, block, 0, s, 0, p); \
    else return launch_pdl(ep_router_kernel<T, JJ>, grid, block, 0, s, 0, p);           \
  }
  EP_ROUTER(1)
  EP_ROUTER(2)
  EP_ROUTER(4)
  EP_ROUTER(8)
  EP_ROUTER(16)
  EP_ROUTER(32)
#undef EP_ROUTER
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_router(const RouterParams& p, int, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP32) return launch_typed<float, false>(p, s);
  if (p.dtype == EP_DTYPE_FP16) return launch_typed<__half, false>(p, s);
  return launch_typed<__nv_bfloat16, false>(p, s);
}

cudaError_t launch_router_bwd(const RouterParams& p, int, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP32) return launch_typed<float, true>(p, s);
  if (p.dtype == EP_DTYPE_FP16) return launch_typed<__half, true>(p, s);
  return launch_typed<__nv_bfloat16, true>(p, s);
}

}  // namespace ep
