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

constexpr int kWarps = 8;

// 16 or 32 bytes, read or written once.
template <int VB>
struct alignas(VB) Vec {
  uint32_t w[VB / 4];
};
template <int VB>
__device__ __forceinline__ Vec<VB> load_once(const Vec<VB>* p) {
  Vec<VB> v;
  if constexpr (VB == 32)
    asm volatile("ld.global.nc.L1::no_allocate.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p));
  else
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "l"(p));
  return v;
}
template <int VB>
__device__ __forceinline__ void store_once(Vec<VB>* p, const Vec<VB>& v) {
  if constexpr (VB == 32)
    asm volatile("st.global.v8.u32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]),
                 "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7]));
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

template <int VB, int U>
__global__ void __launch_bounds__(kWarps * 32) ep_dispatch_f8_kernel(const RowParams p, const uint4* scales, uint4* recv_scales) {
  using V = Vec<VB>;
  pdl_wait();
  const Header head = load_header(p);
  if (!header_ok(head, p)) return;
  const int lane = threadIdx.x & 31;
  const int row = p.rowbytes / VB, srow = scale_columns(p.rowbytes) / 4;  // vectors
  const int pieces = (row + 32 * U - 1) / (32 * U);
  const V* src = static_cast<const V*>(p.src);
  V* dst = static_cast<V*>(p.dst);
  const long long tokens = static_cast<long long>(p.T) * pieces, total = tokens + head.npad;
  for (long long i = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < total; i += static_cast<long long>(gridDim.x) * kWarps) {
    if (i >= tokens) {
      const int to = p.pad_list[i - tokens];
      if (static_cast<unsigned>(to) >= static_cast<unsigned>(p.R)) continue;
      const V zero = {};
      for (int v = lane; v < row; v += 32) store_once(dst + static_cast<long long>(to) * row + v, zero);
      for (int v = lane; v < srow; v += 32) recv_scales[static_cast<long long>(to) * srow + v] = make_uint4(0, 0, 0, 0);
      if (lane == 0) p.w_out[to] = 0.0f;
      continue;
    }
    const int t = static_cast<int>(i / pieces), piece = static_cast<int>(i - static_cast<long long>(t) * pieces);
    // The token's receive rows, one a lane; -1 where a route is masked.
    const int slot = lane < p.K ? __ldg(p.slot + static_cast<long long>(t) * p.K + lane) : -1;
    const int v0 = piece * 32 * U + lane;
    V v[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (v0 + 32 * j < row) v[j] = load_once(src + static_cast<long long>(t) * row + v0 + 32 * j);
    for (int k = 0; k < p.K; ++k) {
      const int to = __shfl_sync(0xffffffffu, slot, k);
      if (static_cast<unsigned>(to) >= static_cast<unsigned>(p.R)) continue;
      V* at = dst + static_cast<long long>(to) * row + v0;
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (v0 + 32 * j < row) store_once(at + 32 * j, v[j]);
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

template <int VB, int U>
cudaError_t launch_vec(const RowParams& p, const float* scales, float* recv_scales, int npad_max, cudaStream_t s) {
  // One item a warp, as far as the padding rows are the tokens' number at most:
  // blocks that follow one another keep the writes streaming (a grid of 8
  // blocks per SM that strides took 110 us, and 16-byte vectors).
  const long long pieces = (p.rowbytes / VB + 32 * U - 1) / (32 * U);
  const long long items = p.T * pieces + std::min<long long>(npad_max, std::max<long long>(p.T, 1024));
  const long long blocks = std::max<long long>(1, std::min<long long>((items + kWarps - 1) / kWarps, 1 << 30));
  return launch_pdl(ep_dispatch_f8_kernel<VB, U>, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, s, 0, p,
                    reinterpret_cast<const uint4*>(scales), reinterpret_cast<uint4*>(recv_scales));
}

}  // namespace

cudaError_t launch_dispatch_f8(const RowParams& p, const float* scales, float* recv_scales, int npad_max, int num_sms, cudaStream_t s) {
  const bool wide = p.rowbytes % 32 == 0 && reinterpret_cast<uintptr_t>(p.src) % 32 == 0 && reinterpret_cast<uintptr_t>(p.dst) % 32 == 0;
  // Few tokens: 512 bytes a warp, so that every SM has some.
  if (static_cast<long long>(p.T) * ((p.rowbytes + 2047) / 2048) < 16LL * num_sms)
    return launch_vec<16, 1>(p, scales, recv_scales, npad_max, s);
  return wide ? launch_vec<32, 2>(p, scales, recv_scales, npad_max, s) : launch_vec<16, 4>(p, scales, recv_scales, npad_max, s);
}

}  // namespace ep
