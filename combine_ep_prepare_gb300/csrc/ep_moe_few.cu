// ep_moe_few.cu -- a whole MoE layer for a few tokens in two kernels.
//
// The first takes the gate's product (and, for 8-bit weights, quantises the
// tokens).  The second chooses the experts in every block by itself, then
// multiplies: a = silu(g) u of the used experts' w13, one wait of the blocks
// for one another, and out = sum over a token's experts of p w2 a.
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "ep_moe_few.cuh"
#include "ep_router.cuh"

namespace ep {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8, kThreads = kWarps * 32;

template <typename G, typename T>
__global__ void __launch_bounds__(kThreads) ep_few_gate_kernel(const FewParams p) {
  __shared__ float part[kWarps][EP_MAX_FEW_TOKENS];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && threadIdx.x < 2) p.hdr[threadIdx.x] = 0;
  if (static_cast<int>(blockIdx.x) < p.E) {
    const int e = blockIdx.x;
    float acc[EP_MAX_FEW_TOKENS];
#pragma unroll
    for (int t = 0; t < EP_MAX_FEW_TOKENS; ++t) acc[t] = 0.0f;
    for (int k = threadIdx.x * 8; k < p.H; k += kThreads * 8) {
      Raw8<G> g;
      float gv[8];
      g.load(static_cast<const G*>(p.gate) + static_cast<long long>(e) * p.H + k);
      g.get(gv);
#pragma unroll
      for (int t = 0; t < EP_MAX_FEW_TOKENS; ++t) {
        if (t < p.T) {
          Raw8<T> x;
          float xv[8];
          x.load(static_cast<const T*>(p.x) + static_cast<long long>(t) * p.H + k);
          x.get(xv);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[t] = fmaf(gv[j], xv[j], acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < EP_MAX_FEW_TOKENS; ++t) {
      if (t < p.T) {
        const float s = route::warp_sum(acc[t]);
        if (lane == 0) part[warp][t] = s;
      }
    }
    __syncthreads();
    if (threadIdx.x < p.T) {
      float s = 0.0f;
      for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
      p.logits[threadIdx.x * p.E + e] = s;
    }
  } else {  // a token's row in 8 bits
    const int t = blockIdx.x - p.E, cols = scale_columns(p.H);
    for (int b = warp * 2; b < cols; b += kWarps * 2) {
      const int k = b * kF8Block + lane * 8;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (k < p.H) {
        Raw8<T> x;
        x.load(static_cast<const T*>(p.x) + static_cast<long long>(t) * p.H + k);
        x.get(v);
      }
      uint2 q;
      const float s = quantize8(v, &q);
      if (k < p.H) *reinterpret_cast<uint2*>(p.xq + static_cast<long long>(t) * p.H + k) = q;
      if ((lane & 15) == 0) p.xs[t * cols + b + (lane >> 4)] = k < p.H ? s : 0.0f;
    }
  }
}

__device__ __forceinline__ float e4m3(uint8_t v) { return static_cast<float>(*reinterpret_cast<const __nv_fp8_e4m3*>(&v)); }

// All blocks of the grid have arrived, and what they wrote before can be read.
// The word was zero when the kernel began.  False after about a second.
__device__ bool grid_wait(unsigned* word, int* status) {
  __shared__ int ok_s;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(word, 1u);
    unsigned v = 0, spins = 0;
    int ok = 1;
    for (;;) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
      if (v >= gridDim.x) break;
      if (++spins > (1u << 20)) {
        ok = 0;
        *status = static_cast<int>(EP_ST_TIMEOUT);
        break;
      }
      __nanosleep(32);
    }
    __threadfence();
    ok_s = ok;
  }
  __syncthreads();
  return ok_s != 0;
}

struct Choice {
  unsigned tokens[EP_MAX_EXPERTS];                       // an expert's tokens, a bit each
  short first[EP_MAX_EXPERTS];                           // the routes of the experts before it
  short used[EP_MAX_FEW_TOKENS * EP_MAX_TOPK];           // experts with a token, ascending
  short expert[EP_MAX_FEW_TOKENS * EP_MAX_TOPK];         // [t][k]
  float weight[EP_MAX_FEW_TOKENS * EP_MAX_TOPK];
  int num_used;
};

template <int J>
__device__ __forceinline__ void choose(const FewParams& p, Choice& c, int warp, int lane) {
  for (int t = warp; t < p.T; t += kWarps) {
    int e;
    float w;
    route::route_token<float, J>(p.router, t, lane, &e, &w);
    if (lane < p.K) {
      c.expert[t * p.K + lane] = static_cast<short>(e);
      c.weight[t * p.K + lane] = w;
      if (e >= 0) atomicOr(&c.tokens[e], 1u << t);
      if (blockIdx.x == 0) {
        p.idx[t * p.K + lane] = e;
        p.w[t * p.K + lane] = w;
      }
    }
  }
}

template <typename T, bool f8>
__global__ void __launch_bounds__(kThreads) ep_few_experts_kernel(const FewParams p) {
  __shared__ Choice c;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < p.E; e += kThreads) c.tokens[e] = 0;
  __syncthreads();
  const int j = (p.E + 31) / 32;
  if (j <= 4) choose<4>(p, c, warp, lane);
  else if (j <= 8) choose<8>(p, c, warp, lane);
  else choose<32>(p, c, warp, lane);
  __syncthreads();
  if (warp == 0) {
    int used = 0, first = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < p.E ? __popc(c.tokens[e]) : 0;
      int sum = n;
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, sum, d);
        if (lane >= d) sum += o;
      }
      const unsigned has = __ballot_sync(kAll, n > 0);
      if (n > 0) {
        c.used[used + __popc(has & ((1u << lane) - 1))] = static_cast<short>(e);
        c.first[e] = static_cast<short>(first + sum - n);
      }
      used += __popc(has);
      first += __shfl_sync(kAll, sum, 31);
    }
    if (lane == 0) c.num_used = used;
  }
  __syncthreads();
  const int hb = f8_blocks(p.H), fb = f8_blocks(p.F);
  const int gw = blockIdx.x * kWarps + warp, warps = gridDim.x * kWarps;
  for (int u = gw; u < c.num_used * p.F; u += warps) {
    const int e = c.used[u / p.F], f = u % p.F;
    const long long wg = (static_cast<long long>(e) * 2 * p.F + f) * p.H, wu = wg + static_cast<long long>(p.F) * p.H;
    int pos = c.first[e];
    for (unsigned left = c.tokens[e]; left; left &= left - 1, ++pos) {
      const int t = __ffs(left) - 1;
      float g = 0.0f, v = 0.0f;
      for (int k = lane; k < p.H; k += 32) {
        if constexpr (f8) {
          const float x = e4m3(p.xq[static_cast<long long>(t) * p.H + k]) * p.xs[t * scale_columns(p.H) + k / 128];
          const uint8_t* w = static_cast<const uint8_t*>(p.w13);
          g = fmaf(x, e4m3(w[wg + k]) * p.s13[(static_cast<long long>(e) * 2 * fb + f / 128) * hb + k / 128], g);
          v = fmaf(x, e4m3(w[wu + k]) * p.s13[(static_cast<long long>(e) * 2 * fb + fb + f / 128) * hb + k / 128], v);
        } else {
          const float x = to_f32(static_cast<const T*>(p.x)[static_cast<long long>(t) * p.H + k]);
          g = fmaf(x, to_f32(static_cast<const T*>(p.w13)[wg + k]), g);
          v = fmaf(x, to_f32(static_cast<const T*>(p.w13)[wu + k]), v);
        }
      }
      g = route::warp_sum(g);
      v = route::warp_sum(v);
      if (lane == 0) {
        const float a = swiglu(g, v);
        p.act[static_cast<long long>(pos) * p.F + f] = f8 ? a : to_f32(from_f32<T>(a));
      }
    }
  }
  if (!grid_wait(reinterpret_cast<unsigned*>(p.hdr + 1), p.hdr)) return;
  for (int h = gw; h < p.H; h += warps) {
    for (int t = 0; t < p.T; ++t) {
      float y = 0.0f;
      for (int k = 0; k < p.K; ++k) {
        const int e = c.expert[t * p.K + k];
        if (e < 0) continue;
        const int pos = c.first[e] + __popc(c.tokens[e] & ((1u << t) - 1));
        const float* a = p.act + static_cast<long long>(pos) * p.F;
        const long long wr = (static_cast<long long>(e) * p.H + h) * p.F;
        float s = 0.0f;
        for (int f0 = 0; f0 < p.F; f0 += 128) {
          float v[4], m = 0.0f;
          for (int i = 0; i < 4; ++i) {
            const int f = f0 + lane * 4 + i;
            v[i] = f < p.F ? __ldcg(a + f) : 0.0f;
            m = max_nan(m, fabsf(v[i]));
          }
          if constexpr (f8) {
            for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, d));
            const BlockScale b = block_scale(m);
            const uint32_t q = e4m3x4(v[0] * b.inv, v[1] * b.inv, v[2] * b.inv, v[3] * b.inv);
            const float scale = b.scale * p.s2[(static_cast<long long>(e) * hb + h / 128) * fb + f0 / 128];
            float part = 0.0f;
            for (int i = 0; i < 4; ++i)
              part = fmaf(e4m3(q >> (8 * i)), e4m3(static_cast<const uint8_t*>(p.w2)[wr + f0 + lane * 4 + i]), part);
            s = fmaf(part, scale, s);
          } else {
            for (int i = 0; i < 4; ++i)
              if (f0 + lane * 4 + i < p.F) s = fmaf(v[i], to_f32(static_cast<const T*>(p.w2)[wr + f0 + lane * 4 + i]), s);
          }
        }
        y = fmaf(c.weight[t * p.K + k], route::warp_sum(s), y);
      }
      if (lane == 0) static_cast<T*>(p.out)[static_cast<long long>(t) * p.H + h] = from_f32<T>(y);
    }
  }
}

template <typename T, bool f8>
cudaError_t launch_experts(const FewParams& p, int num_sms, cudaStream_t s) {
  return launch_pdl_ex(ep_few_experts_kernel<T, f8>, dim3(num_sms), dim3(kThreads), 0, s, 0, true, p);
}

template <typename T>
cudaError_t launch_typed(const FewParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(p.E + (p.f8 ? p.T : 0)), block(kThreads);
  const cudaError_t e = p.gate_dtype == EP_DTYPE_FP32   ? launch_pdl(ep_few_gate_kernel<float, T>, grid, block, 0, s, 0, p)
                        : p.gate_dtype == EP_DTYPE_FP16 ? launch_pdl(ep_few_gate_kernel<__half, T>, grid, block, 0, s, 0, p)
                                                        : launch_pdl(ep_few_gate_kernel<__nv_bfloat16, T>, grid, block, 0, s, 0, p);
  if (e != cudaSuccess) return e;
  return p.f8 ? launch_experts<T, true>(p, num_sms, s) : launch_experts<T, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_moe_few(const FewParams& p, int num_sms, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP16) return launch_typed<__half>(p, num_sms, s);
  return launch_typed<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace ep
