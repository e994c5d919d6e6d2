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
#include "ep_experts.cuh"

namespace ep {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;  // one for each of an SM's schedulers

template <typename T>
__device__ __forceinline__ float logit(const void* p, long long i) { return to_f32(static_cast<const T*>(p)[i]); }

// Unsigned key in the order of v; 0 for -inf and NaN.  Adding +0 makes -0 and
// +0 the same key.
__device__ __forceinline__ unsigned key_of(float v) {
  if (!(v > -INFINITY)) return 0;
  const unsigned u = __float_as_uint(v + 0.0f);
  return u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// 1 / (1 + exp(-z)), the reciprocal rounded correctly, as a division would be.
__device__ __forceinline__ float sigmoidf(float z) { return __frcp_rn(1.0f + expf(-z)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// exp(z - m), 0 where the logit cannot be chosen.  A largest logit of +inf
// makes this NaN, the sum over it and so all weights of the row: a sum is
// compared with 0 alone, which only a row without a choice has.
__device__ __forceinline__ float exp_or_0(float z, float m) { return z > -INFINITY ? expf(z - m) : 0.0f; }

// This lane's J logits from expert lane J on; -inf past the last.
template <typename T, int J>
__device__ __forceinline__ void load_run(const RouterParams& p, long long row, int lane, float (&z)[J]) {
  constexpr int kVec = 16 / sizeof(T) < J ? 16 / sizeof(T) : J;  // elements per load
  const T* at = static_cast<const T*>(p.logits) + row + lane * J;
  if (kVec > 1 && p.E % kVec == 0 && reinterpret_cast<uintptr_t>(p.logits) % (kVec * sizeof(T)) == 0) {
#pragma unroll
    for (int j = 0; j < J; j += kVec) {
      alignas(16) T v[kVec];
      if (lane * J + j < p.E) {
        if constexpr (kVec * sizeof(T) == 16) *reinterpret_cast<uint4*>(v) = __ldg(reinterpret_cast<const uint4*>(at + j));
        else if constexpr (kVec * sizeof(T) == 8) *reinterpret_cast<uint2*>(v) = __ldg(reinterpret_cast<const uint2*>(at + j));
        else if constexpr (kVec * sizeof(T) == 4) *reinterpret_cast<uint32_t*>(v) = __ldg(reinterpret_cast<const uint32_t*>(at + j));
        else v[0] = at[j];
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) z[j + i] = lane * J + j < p.E ? to_f32(v[i]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j) z[j] = lane * J + j < p.E ? to_f32(at[j]) : -INFINITY;
  }
}

// A group's rank from its two largest keys (0: none).  Half the sum of the
// two: the same order, and two logits at the type's lowest value do not
// overflow to -inf.
__device__ __forceinline__ unsigned group_key(unsigned best, unsigned second) {
  if (best == 0) return 0;
  const float f = value_of(best);
  return key_of(0.5f * f + 0.5f * (second != 0 ? value_of(second) : f));
}

template <typename T, int J>
__global__ void __launch_bounds__(kWarps * 32) ep_router_kernel(const RouterParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const long long row = static_cast<long long>(t) * p.E;
  unsigned key[J];
  // Softmax over all experts: the largest logit and the sum of exponentials.
  float zmax = 0.0f, zsum = 1.0f;
  {
    float z[J];
    load_run<T, J>(p, row, lane, z);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float v = z[j];
      if (p.sigmoid) {
        v = sigmoidf(z[j]);
        const int e = lane * J + j;
        if (p.bias != nullptr && e < p.E) v += __ldg(p.bias + e);
      }
      key[j] = z[j] > -INFINITY ? key_of(v) : 0;
    }
    if (!p.sigmoid && !p.normalize) {
      unsigned m = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) m = max(m, key[j]);
      m = __reduce_max_sync(kAll, m);
      zmax = m ? value_of(m) : 0.0f;
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j) s += exp_or_0(z[j], zmax);
      zsum = warp_sum(s);
    }
  }
  // This lane's best two (of equal ones the lower index first); more are
  // looked for only when a lane has had two chosen.
  unsigned a = 0, b = 0;
  int at = 0, bt = 0;
  auto best_two = [&]() {
    a = b = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool over_a = key[j] > a, over_b = key[j] > b;
      b = over_a ? a : over_b ? key[j] : b;
      bt = over_a ? at : over_b ? j : bt;
      a = over_a ? key[j] : a;
      at = over_a ? j : at;
    }
  };
  best_two();
  if (p.groups > 1) {
    const int per = p.E / p.groups;
    const int span = per / J;  // lanes of a group, where groups are runs of whole lanes
    unsigned gkey = 0;         // one lane of each group, ascending: its rank
    int shift = 0;             // log2 of the lanes between those
    const bool whole = per % J == 0 && (span & (span - 1)) == 0;
    if (whole) {
      unsigned x = a, y = b;
      for (int d = 1; d < span; d <<= 1, ++shift) {
        const unsigned ox = __shfl_xor_sync(kAll, x, d), oy = __shfl_xor_sync(kAll, y, d);
        y = max(min(x, ox), max(y, oy));
        x = max(x, ox);
      }
      if ((lane & (span - 1)) == 0) gkey = group_key(x, y);
    } else {
      for (int g = 0; g < p.groups; ++g) {
        unsigned x = 0, y = 0;  // this lane's two best of group g
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int e = lane * J + j;
          if (e >= g * per && e < (g + 1) * per) {
            y = max(y, min(x, key[j]));
            x = max(x, key[j]);
          }
        }
        const unsigned best = __reduce_max_sync(kAll, x);
        const unsigned holders = __ballot_sync(kAll, x == best);
        // The second best: the best again where two lanes hold it, else the
        // best of the other lanes' first and the holder's second.
        const unsigned second = __reduce_max_sync(kAll, (holders & (holders - 1)) ? best : (x == best ? y : x));
        if (lane == g) gkey = group_key(best, second);
      }
    }
    unsigned keep = 0;  // bit of each kept group's lane; of equal ranks the lowest
    for (int i = 0; i < p.kept; ++i) {
      const unsigned best = __reduce_max_sync(kAll, gkey);
      if (best == 0) break;
      const unsigned holders = __ballot_sync(kAll, gkey == best), lowest = holders & (0u - holders);
      keep |= lowest;
      if (lowest >> lane & 1) gkey = 0;
    }
    if (whole) {
      if (!(keep >> (lane >> shift << shift) & 1)) a = b = 0;
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int e = lane * J + j;
        if (e < p.E && !(keep >> (e / per) & 1)) key[j] = 0;
      }
      best_two();
    }
  }
  int mine = -1, had = 0;  // lane k: the k-th choice; how many of this lane's were chosen
  for (int k = 0; k < p.K; ++k) {
    const unsigned top = __reduce_max_sync(kAll, a);
    if (top == 0) break;
    const int l = __ffs(__ballot_sync(kAll, a == top)) - 1;
    const int e = l * J + __shfl_sync(kAll, at, l);
    if (lane == k) mine = e;
    if (lane == l) {
      if (++had == 1) {
        a = b;
        at = bt;
      } else {
        // The best after (top, at) in the order of the choice.
        const int last = at;
        a = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool left = key[j] < top || (key[j] == top && j > last);
          if (left && key[j] > a) {
            a = key[j];
            at = j;
          }
        }
      }
    }
  }
  // Weights: lane k has the k-th choice's.
  const float zk = mine >= 0 ? logit<T>(p.logits, row + mine) : -INFINITY;
  float w;
  if (p.sigmoid) {
    w = mine >= 0 ? sigmoidf(zk) : 0.0f;
    if (p.normalize) {
      const float total = warp_sum(w);
      w = total > 0.0f ? w / total : 0.0f;
    }
  } else if (p.normalize) {
    const float m = __shfl_sync(kAll, zk, 0);  // the first choice has the largest logit
    w = exp_or_0(zk, m);
    const float total = warp_sum(w);
    w = total != 0.0f ? w / total : 0.0f;
  } else {
    w = exp_or_0(zk, zmax) / (zsum != 0.0f ? zsum : 1.0f);
  }
  if (lane < p.K) {
    p.idx[static_cast<long long>(t) * p.K + lane] = mine;
    p.w[static_cast<long long>(t) * p.K + lane] = w * p.scale;
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
