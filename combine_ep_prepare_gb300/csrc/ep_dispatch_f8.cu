// ep_dispatch_f8.cu -- dispatch of 8-bit rows with their scales and weights.
//
// A warp takes 2 KB of a token's row (four 16-byte vectors a lane), reads them
// once and writes them to the token's K receive rows; the warp of a row's first
// piece takes the scales and the weights along.  Padding rows are zeroed by the
// warps that are left.  Bound by the writes: 8,192 tokens of 7168 to 65,536 rows
// are 487 MB.  (The 16-bit scatter, once for the rows and once for the scales,
// took 141 us with the quantisation before it; its second pass moves 224 bytes
// a row.)
#include <algorithm>

#include "ep_f8.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8, kVecs = 4;

__global__ void __launch_bounds__(kWarps * 32) ep_dispatch_f8_kernel(const RowParams p, const uint4* scales, uint4* recv_scales) {
  pdl_wait();
  const Header head = load_header(p);
  if (!header_ok(head, p)) return;
  const int lane = threadIdx.x & 31;
  const int row = p.rowbytes / 16, srow = scale_columns(p.rowbytes) / 4;  // vectors
  const int pieces = (row + 32 * kVecs - 1) / (32 * kVecs);
  const uint4* src = static_cast<const uint4*>(p.src);
  uint4* dst = static_cast<uint4*>(p.dst);
  const long long tokens = static_cast<long long>(p.T) * pieces, total = tokens + head.npad;
  for (long long i = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < total; i += static_cast<long long>(gridDim.x) * kWarps) {
    if (i >= tokens) {
      const int to = p.pad_list[i - tokens];
      if (static_cast<unsigned>(to) >= static_cast<unsigned>(p.R)) continue;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      for (int v = lane; v < row; v += 32) dst[static_cast<long long>(to) * row + v] = zero;
      for (int v = lane; v < srow; v += 32) recv_scales[static_cast<long long>(to) * srow + v] = zero;
      if (lane == 0) p.w_out[to] = 0.0f;
      continue;
    }
    const int t = static_cast<int>(i / pieces), piece = static_cast<int>(i - static_cast<long long>(t) * pieces);
    // The token's receive rows, one a lane; -1 where a route is masked.
    const int slot = lane < p.K ? __ldg(p.slot + static_cast<long long>(t) * p.K + lane) : -1;
    const int v0 = piece * 32 * kVecs + lane;
    uint4 v[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      if (v0 + 32 * j < row) v[j] = __ldg(src + static_cast<long long>(t) * row + v0 + 32 * j);
    for (int k = 0; k < p.K; ++k) {
      const int to = __shfl_sync(0xffffffffu, slot, k);
      if (static_cast<unsigned>(to) >= static_cast<unsigned>(p.R)) continue;
      uint4* at = dst + static_cast<long long>(to) * row + v0;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (v0 + 32 * j < row) at[32 * j] = v[j];
    }
    if (piece == 0) {
      for (int s = lane; s < srow; s += 32) {
        const uint4 x = __ldg(scales + static_cast<long long>(t) * srow + s);
        for (int k = 0; k < p.K; ++k) {
          const int to = __ldg(p.slot + static_cast<long long>(t) * p.K + k);
          if (static_cast<unsigned>(to) < static_cast<unsigned>(p.R)) recv_scales[static_cast<long long>(to) * srow + s] = x;
        }
      }
      if (static_cast<unsigned>(slot) < static_cast<unsigned>(p.R)) p.w_out[slot] = __ldg(p.w_in + static_cast<long long>(t) * p.K + lane);
    }
  }
}

}  // namespace

cudaError_t launch_dispatch_f8(const RowParams& p, const float* scales, float* recv_scales, int npad_max, int num_sms, cudaStream_t s) {
  const long long pieces = (p.rowbytes / 16 + 32 * kVecs - 1) / (32 * kVecs);
  const long long warps = p.T * pieces + npad_max;
  const long long blocks = std::max<long long>(1, std::min<long long>((warps + kWarps - 1) / kWarps, 8LL * num_sms));
  return launch_pdl(ep_dispatch_f8_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, s, 0, p,
                    reinterpret_cast<const uint4*>(scales), reinterpret_cast<uint4*>(recv_scales));
}

}  // namespace ep
