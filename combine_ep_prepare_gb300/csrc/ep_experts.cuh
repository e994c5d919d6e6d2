// ep_experts.cuh -- declarations of the expert products, the 4-bit products
// and the router, shared by their translation units.
//
// A group ("expert") e of a prepared handle has c_e rows from off_e on in a
// receive buffer of R rows, its block padded to p_e rows.  The products read
// rows [off_e, off_e + c_e) alone and write rows [off_e, off_e + p_e): zeros
// in the padding.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ep_internal.cuh"

namespace ep {

// Access to the library's state for the calls outside ep_api.cu (defined there).
ep_status_t api_fail(ep_status_t code, const char* msg);
ep_status_t api_cuda_fail(cudaError_t e, const char* where);
// The layer of a handle whose receive rows hold experts of this rank: single
// buffer or expert-major sharded; a rank-major layer is refused.
ep_status_t api_expert_layer(const ep_handle_t& h, const LayerInfo** out);
ep_status_t api_device(int* num_sms);
void api_count_launches(int n);

// Which product.  "rows" are receive rows, "wide" the features.
enum ProductKind {
  kProdFwd = 0,        // out[r][n]   = sum_k a[r][k] w[e][n][k]
  kProdFwdSwiglu = 1,  // the same with n over 2F; pre (may be null) and act[r][F]
  kProdDgrad = 2,      // out[r][k]   = sum_n a[r][n] w[e][n][k]
  kProdDgradSwiglu = 3,  // the same, then through the activation: out[r][2F] from pre
  kProdWgrad = 4       // out[e][n][k] (+)= sum over the expert's rows a[r][n] b[r][k]
};

struct ProductParams {
  int* hdr;
  const int* counts;   // c_e
  const int* offsets;  // off_e, e = 0..E
  int E;               // experts whose rows the buffer holds
  int R;               // receive rows
  int kind;            // ProductKind
  int dtype;           // of a, b / w, pre, and of out unless out_f32
  int out_f32;         // wgrad: out is float32
  int accumulate;      // wgrad: add to out
  int N;               // weight rows per expert (2F for the gated pair)
  int K;               // weight columns
  const void* a;       // [R][K] forward, [R][N] gradients
  const void* b;       // weights [E][N][K]; wgrad: rows [R][K]
  const void* pre;     // dgrad_swiglu: [R][2K]
  void* out;
  void* out2;          // fwd_swiglu: pre [R][N] or null
};

// The header of a prepared handle with usable blocks.
__device__ __forceinline__ bool blocks_ok(const int* hdr, int R) {
  return hdr[kHdrMagic] == kPreparedMagic &&
         !(hdr[kHdrStatus] & (EP_ST_OVERFLOW | EP_ST_COUNTS_MISMATCH)) && hdr[kHdrP] <= R;
}

// Inclusive scan of v over the block's threads; `part` holds 32 ints.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  int add = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w)
    if (w < warp) add += part[w];
  __syncthreads();
  return v + add;
}

// cum[e] = blocks of `tile` rows of the experts before e, e = 0..E, over the
// padded rows.  All THREADS threads call it; `part` holds 32 ints.
template <int THREADS>
__device__ __forceinline__ void scan_row_tiles(const int* offsets, int E, int tile, int* cum, int* part) {
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += THREADS) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int rows = e < E ? offsets[e + 1] - offsets[e] : 0;
    const int v = block_scan<THREADS>((rows + tile - 1) / tile, part);
    if (e < E) cum[e + 1] = base + v;
    if (threadIdx.x == THREADS - 1) part[0] = v;
    __syncthreads();
    base += part[0];
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[0] = 0;
  __syncthreads();
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// silu(gate) * up and its two derivatives times da, in float32.  For a very
// negative gate exp(-gate) is infinite and gate / (1 + inf) is -0; the
// derivative's gate * (1 - sg) times sg = 0 stays finite too.
__device__ __forceinline__ float swiglu(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }
__device__ __forceinline__ void swiglu_bwd(float gate, float up, float da, float* dgate, float* dup) {
  const float sg = 1.0f / (1.0f + expf(-gate));
  *dgate = da * up * sg * (1.0f + gate * (1.0f - sg));
  *dup = da * gate * sg;
}

// Products of float32 rows on the CUDA cores.
cudaError_t launch_product_simt(const ProductParams& p, int num_sms, cudaStream_t s);
// Products of bf16 and fp16 rows on the tensor cores.
cudaError_t launch_product_tc(const ProductParams& p, int num_sms, cudaStream_t s);

struct W4Params {
  int* hdr;
  const int* counts;
  const int* offsets;
  int E, R;
  int dtype;
  int N, K, group;
  int swiglu;          // N = 2F rows of gate, then up; out [R][F]
  const void* x;       // [R][K]
  const uint8_t* wq;   // [E][N][K/2]
  const void* scales;  // [E][N][K/group]
  void* out;
};
cudaError_t launch_w4(const W4Params& p, int num_sms, cudaStream_t s);

struct RouterParams {
  int T, E, K, groups, kept;
  int sigmoid, normalize, dtype;
  float scale;
  const void* logits;   // [T][E]
  const float* bias;    // [E] or null
  long long* idx;       // [T][K]
  float* w;             // [T][K]
  const float* grad;    // backward: [T][K]
  void* grad_logits;    // [T][E]
};
cudaError_t launch_router(const RouterParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_router_bwd(const RouterParams& p, int num_sms, cudaStream_t s);

}  // namespace ep
