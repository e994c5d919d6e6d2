// ep_products_f8.cu -- products grouped by expert of e4m3 rows and weights
// with a scale for each block of 128.
//
//   forward  out[r][n] = sum_b as[r][b] ws[n/128][b] sum_{k in b} a[r][k] w[n][k]
//   dgrad    out[r][k] = sum_b as[r][b] ws[b][k/128] sum_{n in b} a[r][n] w[n][k]
//
// A block takes one row's 128 features, a thread one of them.
#include <cuda_fp8.h>

#include "ep_f8.cuh"

namespace ep {
namespace {

__device__ __forceinline__ float e4m3(uint8_t v) {
  return static_cast<float>(*reinterpret_cast<const __nv_fp8_e4m3*>(&v));
}

template <typename T, int kind>
__global__ void __launch_bounds__(128) ep_product_f8_kernel(const F8Params p) {
  __shared__ float part[4];
  pdl_wait();
  if (!blocks_ok(p.hdr, p.R)) return;
  constexpr bool fwd = kind == kProdFwd || kind == kProdFwdSwiglu;
  const int red = fwd ? p.K : p.N, kb = f8_blocks(p.K), nb = f8_blocks(p.N);
  const int cols = kind == kProdFwd ? p.N : kind == kProdFwdSwiglu ? p.N / 2 : p.K;
  const int c = blockIdx.y * 128 + threadIdx.x;
  int e = 0;
  for (int r = blockIdx.x; r < p.hdr[kHdrP]; r += gridDim.x) {
    while (r >= p.offsets[e + 1]) ++e;
    const bool live = r - p.offsets[e] < p.counts[e];
    const uint8_t* w = p.w + static_cast<long long>(e) * p.N * p.K;
    const float* ws = p.ws + static_cast<long long>(e) * nb * kb;
    const uint8_t* a = p.a + static_cast<long long>(r) * red;
    const float* as = p.as + static_cast<long long>(r) * scale_columns(red);
    float s0 = 0.0f, s1 = 0.0f;
    if (live && c < cols) {
      for (int b = 0; b < f8_blocks(red); ++b) {
        float t0 = 0.0f, t1 = 0.0f;
        for (int i = b * 128; i < min(red, b * 128 + 128); ++i) {
          const float x = e4m3(a[i]);
          t0 = fmaf(x, e4m3(fwd ? w[static_cast<long long>(c) * p.K + i] : w[static_cast<long long>(i) * p.K + c]), t0);
          if (kind == kProdFwdSwiglu) t1 = fmaf(x, e4m3(w[static_cast<long long>(c + cols) * p.K + i]), t1);
        }
        s0 = fmaf(t0, as[b] * (fwd ? ws[c / 128 * kb + b] : ws[b * kb + c / 128]), s0);
        if (kind == kProdFwdSwiglu) s1 = fmaf(t1, as[b] * ws[(c + cols) / 128 * kb + b], s1);
      }
    }
    const long long at = static_cast<long long>(r) * cols + c;
    if constexpr (kind == kProdFwdSwiglu) {
      const float act = swiglu(s0, s1);
      if (c < cols) {
        if (p.pre != nullptr) {
          static_cast<T*>(p.pre)[static_cast<long long>(r) * p.N + c] = from_f32<T>(s0);
          static_cast<T*>(p.pre)[static_cast<long long>(r) * p.N + cols + c] = from_f32<T>(s1);
        }
        if (p.out != nullptr) static_cast<T*>(p.out)[at] = from_f32<T>(act);
      }
      if (p.q != nullptr) {
        float m = c < cols ? fabsf(act) : 0.0f;
        for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        const BlockScale s = block_scale(max_nan(max_nan(part[0], part[1]), max_nan(part[2], part[3])));
        __syncthreads();
        if (c < cols) p.q[at] = live ? static_cast<uint8_t>(e4m3x2(act * s.inv, 0.0f)) : 0;
        const long long sat = static_cast<long long>(r) * scale_columns(cols);
        if (threadIdx.x == 0) p.qs[sat + blockIdx.y] = live ? s.scale : 0.0f;
        if (blockIdx.y == 0 && threadIdx.x >= f8_blocks(cols) && threadIdx.x < scale_columns(cols)) p.qs[sat + threadIdx.x] = 0.0f;
      }
    } else if (c < cols) {
      if constexpr (kind == kProdDgradSwiglu) {
        const long long i = static_cast<long long>(r) * 2 * cols + c;
        float dg = 0.0f, du = 0.0f;
        if (live)
          swiglu_bwd(to_f32(static_cast<const T*>(p.pre_in)[i]), to_f32(static_cast<const T*>(p.pre_in)[i + cols]), s0, &dg, &du);
        static_cast<T*>(p.out)[i] = from_f32<T>(dg);
        static_cast<T*>(p.out)[i + cols] = from_f32<T>(du);
      } else {
        static_cast<T*>(p.out)[at] = from_f32<T>(s0);
      }
    }
  }
}

template <typename T>
cudaError_t launch_typed(const F8Params& p, cudaStream_t s) {
  const int cols = p.kind == kProdFwd ? p.N : p.kind == kProdFwdSwiglu ? p.N / 2 : p.K;
  const dim3 grid(p.R < 4096 ? p.R : 4096, (cols + 127) / 128), block(128);
  switch (p.kind) {
    case kProdFwd: return launch_pdl(ep_product_f8_kernel<T, kProdFwd>, grid, block, 0, s, 0, p);
    case kProdFwdSwiglu: return launch_pdl(ep_product_f8_kernel<T, kProdFwdSwiglu>, grid, block, 0, s, 0, p);
    case kProdDgrad: return launch_pdl(ep_product_f8_kernel<T, kProdDgrad>, grid, block, 0, s, 0, p);
    default: return launch_pdl(ep_product_f8_kernel<T, kProdDgradSwiglu>, grid, block, 0, s, 0, p);
  }
}

}  // namespace

cudaError_t launch_product_f8(const F8Params& p, int, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP16) return launch_typed<__half>(p, s);
  return launch_typed<__nv_bfloat16>(p, s);
}

}  // namespace ep
