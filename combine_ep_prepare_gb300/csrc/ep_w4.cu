// ep_w4.cu -- products of a few rows per expert with 4-bit weights.
//
// w[e][n][k] = scales[e][n][k / group] * (q - 8), q the unsigned nibble k of
// row n (low nibble of a byte: even k).  out[r][n] = sum_k x[r][k] w[e][n][k]
// for the rows of expert e, or silu(gate) * up of the two halves of n.
#include "ep_experts.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 8;  // rows per pass over the weights

// One warp per output feature: lanes stride over the reduction eight weights
// at a time, kRows receive rows share the unpacked weights.
template <typename T, bool gated>
__global__ void __launch_bounds__(kWarps * 32) ep_w4_kernel(const W4Params p) {
  pdl_wait();
  if (!blocks_ok(p.hdr, p.R)) return;
  const int lane = threadIdx.x & 31;
  const int cols = gated ? p.N / 2 : p.N;
  const long long total = static_cast<long long>(p.E) * cols;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  for (long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < total;
       item += static_cast<long long>(gridDim.x) * kWarps) {
    const int e = static_cast<int>(item / cols), n = static_cast<int>(item - static_cast<long long>(e) * cols);
    const long long off = p.offsets[e];
    const int cnt = p.counts[e], rows = p.offsets[e + 1] - p.offsets[e];
    for (int r0 = 0; r0 < cnt; r0 += kRows) {
      float acc[2][kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc[0][i] = acc[1][i] = 0.0f;
      for (int k = lane * 8; k < p.K; k += 256) {
#pragma unroll
        for (int h = 0; h < (gated ? 2 : 1); ++h) {
          const long long wr = static_cast<long long>(e) * p.N + n + (h ? cols : 0);
          const unsigned q = *reinterpret_cast<const unsigned*>(p.wq + wr * (p.K / 2) + k / 2);
          const float s = to_f32(static_cast<const T*>(p.scales)[wr * (p.K / p.group) + k / p.group]);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            if (r0 + i >= cnt) break;
            const T* xr = x + (off + r0 + i) * p.K + k;
            float d = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              d = fmaf(to_f32(xr[j]), static_cast<float>(static_cast<int>((q >> (4 * j)) & 15) - 8), d);
            acc[h][i] = fmaf(s, d, acc[h][i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          acc[0][i] += __shfl_xor_sync(0xffffffffu, acc[0][i], d);
          if (gated) acc[1][i] += __shfl_xor_sync(0xffffffffu, acc[1][i], d);
        }
        if (lane == 0 && r0 + i < cnt)
          out[(off + r0 + i) * cols + n] = from_f32<T>(gated ? swiglu(acc[0][i], acc[1][i]) : acc[0][i]);
      }
    }
    for (int r = cnt + lane; r < rows; r += 32) out[(off + r) * cols + n] = from_f32<T>(0.0f);
  }
}

}  // namespace

cudaError_t launch_w4(const W4Params& p, int num_sms, cudaStream_t s) {
  const dim3 grid(num_sms * 4), block(kWarps * 32);
  if (p.dtype == EP_DTYPE_FP16)
    return p.swiglu ? launch_pdl(ep_w4_kernel<__half, true>, grid, block, 0, s, 0, p)
                    : launch_pdl(ep_w4_kernel<__half, false>, grid, block, 0, s, 0, p);
  return p.swiglu ? launch_pdl(ep_w4_kernel<__nv_bfloat16, true>, grid, block, 0, s, 0, p)
                  : launch_pdl(ep_w4_kernel<__nv_bfloat16, false>, grid, block, 0, s, 0, p);
}

}  // namespace ep
