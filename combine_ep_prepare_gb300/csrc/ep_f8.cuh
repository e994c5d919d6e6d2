// ep_f8.cuh -- 8-bit rows: what the norm, the quantisation, the products in
// e4m3 and a few tokens' layer share.
//
// A row of n features is held as e4m3 with one float32 scale for each 128 of
// them, a row of scales padded to scale_columns(n) floats.  A block's largest
// magnitude m (at least kLeastMax) becomes 448, the type's largest value.
#pragma once

#include "ep_experts.cuh"

namespace ep {

constexpr int kF8Block = 128;
constexpr float kF8Max = 448.0f;
// Below it 448 / m would leave float32's range on the way to tiny blocks.
constexpr float kLeastMax = 7.8886090522101181e-31f;  // 2^-100

__host__ __device__ __forceinline__ int f8_blocks(int n) { return (n + kF8Block - 1) / kF8Block; }
__host__ __device__ __forceinline__ int scale_columns(int n) { return (f8_blocks(n) + 3) & ~3; }

// The larger magnitude; NaN when either is (fmaxf would drop it, and with it a
// block's only sign of a NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct BlockScale {
  float scale, inv;
};
__device__ __forceinline__ BlockScale block_scale(float m) {
  m = max_nan(m, kLeastMax);
  return {__fdiv_rn(m, kF8Max), __fdiv_rn(kF8Max, m)};
}

// Two values to e4m3, nearest even, saturating; the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | e4m3x2(c, d) << 16;
}

// Eight elements from a 16-byte boundary (float32: 32 bytes of it).
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32(h[i]);
}
template <typename T>
struct Raw8 {
  uint4 u;
  __device__ __forceinline__ void load(const T* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_rw(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8<T>(u, v); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_rw(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  alignas(16) T h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = from_f32<T>(v[i]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sixteen lanes hold a block of 128, eight elements each (zeros past the row's
// end): quantised, and the scale in every one of them.  All 32 lanes call it.
__device__ __forceinline__ float quantize8(const float (&v)[8], uint2* q) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  const BlockScale s = block_scale(m);
  q->x = e4m3x4(v[0] * s.inv, v[1] * s.inv, v[2] * s.inv, v[3] * s.inv);
  q->y = e4m3x4(v[4] * s.inv, v[5] * s.inv, v[6] * s.inv, v[7] * s.inv);
  return s.scale;
}

struct NormParams {
  int T, H, dtype;
  float eps;
  const void* x;
  const void* residual;  // or null
  const void* weight;
  void* sum;             // or null
  void* y;               // or null
  uint8_t* q;            // or null
  float* scales;
  // backward: x is h
  const void* dy;
  const void* dsum;      // or null
  void* dh;
  float* dw;
  int accumulate;
  float* partial;        // [parts][H]
};
// Blocks of the backward pass, each with one row of partial sums.
int norm_bwd_parts(long long T, long long H);
cudaError_t launch_norm(const NormParams& p, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s);

struct QuantParams {
  const int* hdr;      // a prepared handle's, or null: all R rows
  const int* counts;
  const int* offsets;
  int E, R, n, dtype;
  const void* x;
  uint8_t* q;
  float* scales;
};
cudaError_t launch_quantize(const QuantParams& p, int num_sms, cudaStream_t s);

struct F8Params {
  int* hdr;
  const int* counts;
  const int* offsets;
  int E, R;
  int kind;               // ProductKind, without wgrad
  int dtype;              // of pre and the 16-bit outputs
  int N, K;               // weight rows (2F for the gated pair) and columns
  const uint8_t* a;       // rows: [R][K] forward, [R][N] gradients
  const float* as;        // their scales
  const uint8_t* w;       // [E][N][K]
  const float* ws;        // [E][blocks of N][blocks of K]
  const void* pre_in;     // dgrad_swiglu: [R][2K]
  void* out;              // fwd_swiglu: act, or null
  void* pre;              // fwd_swiglu: [R][N], or null
  uint8_t* q;             // fwd_swiglu: act in 8 bits, or null
  float* qs;
};
cudaError_t launch_product_f8(const F8Params& p, int num_sms, cudaStream_t s);

}  // namespace ep
