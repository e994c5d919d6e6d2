// ep_products.cu -- products grouped by expert on the CUDA cores.
//
// For every expert e with rows [off_e, off_e + c_e):
//   forward   out[r][n] = sum_k a[r][k] w[e][n][k]
//   dgrad     out[r][k] = sum_n a[r][n] w[e][n][k]
//   wgrad     out[e][n][k] (+)= sum_r a[r][n] b[r][k]
// with the gated activation silu(gate) * up, or its derivative, applied to the
// float32 sums before the one rounding.  Sums are float32 fused multiply-adds
// in ascending order of the reduction.
#include "ep_experts.cuh"

namespace ep {
namespace {

constexpr int kTile = 128;   // output tile, rows and columns
constexpr int kStep = 16;    // reduction elements per step
constexpr int kThreads = 256;
constexpr int kPad = 4;      // shared-memory row padding against bank conflicts

// Eight consecutive elements as float32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    alignas(8) T e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(e);
  }
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = to_f32(p[i]);
}

// One operand's share of a step: 8 elements per thread of a kTile x kStep slab.
// kc: the reduction index is the contiguous one.
template <typename T, bool kc>
struct Slab {
  float v[8];
  // base: element (0, 0); ld: elements between rows; mn / k limits.
  __device__ __forceinline__ void load(const T* base, long long ld, int mn_lim, int k0, int k_lim) {
    const int t = threadIdx.x;
    const int mn = kc ? t >> 1 : (t & 15) * 8;
    const int k = k0 + (kc ? (t & 1) * 8 : t >> 4);
    if (mn < mn_lim && k < k_lim) {
      load8(kc ? base + mn * ld + k : base + k * ld + mn, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  }
  __device__ __forceinline__ void store(float (*s)[kTile + kPad]) const {
    const int t = threadIdx.x;
    if constexpr (kc) {
      const int mn = t >> 1, k = (t & 1) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k + i][mn] = v[i];
    } else {
      const int mn = (t & 15) * 8, k = t >> 4;
      *reinterpret_cast<float4*>(&s[k][mn]) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(&s[k][mn + 4]) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
};

// A 128 x 128 tile per block, 8 x 8 sums per thread (rows and columns in two
// runs of four, 64 apart, so that a warp's shared-memory reads of four floats
// do not collide), the next step's loads in flight while the present one is
// multiplied.  In the gated forward the tile's columns are 64 gate and 64 up
// columns of the same features, so that one thread holds both.
template <typename T, int kind>
__global__ void __launch_bounds__(kThreads) ep_product_simt_kernel(const ProductParams p) {
  constexpr bool rows_out = kind != kProdWgrad;
  constexpr bool a_kc = rows_out;
  constexpr bool b_kc = kind == kProdFwd || kind == kProdFwdSwiglu;
  __shared__ __align__(16) float sa[2][kStep][kTile + kPad];
  __shared__ __align__(16) float sb[2][kStep][kTile + kPad];
  __shared__ int cum[EP_MAX_EXPERTS + 1];
  __shared__ int part[32];
  pdl_wait();
  if (!blocks_ok(p.hdr, p.R)) return;
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
  const T* a = static_cast<const T*>(p.a);
  const T* b = static_cast<const T*>(p.b);
  const int F = p.N / 2;
  constexpr int cols_per_tile = kind == kProdFwdSwiglu ? kTile / 2 : kTile;
  const int cols = kind == kProdFwd ? p.N : kind == kProdFwdSwiglu ? F : p.K;
  const int ntiles = (cols + cols_per_tile - 1) / cols_per_tile;
  const int wrow_tiles = (p.N + kTile - 1) / kTile;  // wgrad
  long long total;
  if constexpr (rows_out) {
    scan_row_tiles<kThreads>(p.offsets, p.E, kTile, cum, part);
    total = static_cast<long long>(cum[p.E]) * ntiles;
  } else {
    total = static_cast<long long>(p.E) * wrow_tiles * ntiles;
  }
  int e = 0;
  for (long long tile = blockIdx.x; tile < total; tile += gridDim.x) {
    int m0, c0, off, cnt, rows;
    if constexpr (rows_out) {
      while (tile >= static_cast<long long>(cum[e + 1]) * ntiles) ++e;
      const int in = static_cast<int>(tile - static_cast<long long>(cum[e]) * ntiles);
      const int mt = cum[e + 1] - cum[e];
      m0 = in % mt * kTile;
      c0 = in / mt * cols_per_tile;
      off = p.offsets[e];
      rows = p.offsets[e + 1] - off;
      cnt = p.counts[e];
    } else {
      const int per = wrow_tiles * ntiles;
      e = static_cast<int>(tile / per);
      const int in = static_cast<int>(tile - static_cast<long long>(e) * per);
      m0 = in % wrow_tiles * kTile;
      c0 = in / wrow_tiles * kTile;
      off = p.offsets[e];
      rows = cnt = p.counts[e];
    }
    // Operands of this tile.
    const long long w0 = static_cast<long long>(e) * p.N * p.K;
    const T *ab, *bb;
    long long ald, bld;
    int a_lim, b_lim, red;
    if constexpr (rows_out) {
      ald = b_kc ? p.K : p.N;
      ab = a + (static_cast<long long>(off) + m0) * ald;
      a_lim = cnt - m0;
      red = b_kc ? p.K : p.N;
      bld = p.K;
      bb = b + w0 + (b_kc ? static_cast<long long>(c0) * p.K : c0);
      b_lim = cols - c0;
    } else {
      ald = p.N;
      ab = a + static_cast<long long>(off) * p.N + m0;
      a_lim = p.N - m0;
      bld = p.K;
      bb = b + static_cast<long long>(off) * p.K + c0;
      b_lim = p.K - c0;
      red = cnt;
    }
    float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;

    Slab<T, a_kc> la;
    Slab<T, b_kc> lb;
    auto load = [&](int k0) {
      la.load(ab, ald, a_lim, k0, red);
      if constexpr (kind == kProdFwdSwiglu) {
        // slab columns 0..63: gate features c0.., 64..127: up features c0..
        const int half = t >> 7;
        lb.load(bb + (half ? (static_cast<long long>(F) - 64) * bld : 0), bld,
                half ? (b_lim < 64 ? b_lim : 64) + 64 : (b_lim < 64 ? b_lim : 64), k0, red);
      } else {
        lb.load(bb, bld, b_lim, k0, red);
      }
    };
    if (a_lim > 0 && red > 0) {
      load(0);
      la.store(sa[0]);
      lb.store(sb[0]);
      __syncthreads();
      int buf = 0;
      for (int k0 = 0; k0 < red; k0 += kStep) {
        const bool more = k0 + kStep < red;
        if (more) load(k0 + kStep);
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
          float ra[8], rb[8];
          *reinterpret_cast<float4*>(ra) = *reinterpret_cast<const float4*>(&sa[buf][k][ty * 4]);
          *reinterpret_cast<float4*>(ra + 4) = *reinterpret_cast<const float4*>(&sa[buf][k][64 + ty * 4]);
          *reinterpret_cast<float4*>(rb) = *reinterpret_cast<const float4*>(&sb[buf][k][tx * 4]);
          *reinterpret_cast<float4*>(rb + 4) = *reinterpret_cast<const float4*>(&sb[buf][k][64 + tx * 4]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(ra[i], rb[j], acc[i][j]);
        }
        if (more) {
          la.store(sa[buf ^ 1]);
          lb.store(sb[buf ^ 1]);
        }
        __syncthreads();
        buf ^= 1;
      }
    }
    // Epilogue: rows m0 + {0, 64} + 4 ty + i.  A padding row's sums are +0
    // (its operand was not read), so it gets zeros without a case of its own,
    // except through the activation's derivative, which reads `pre`.
    const int m_lim = rows_out ? rows - m0 : p.N - m0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = (i >> 2) * 64 + ty * 4 + (i & 3);
      if (m >= m_lim) continue;
      if constexpr (kind == kProdFwdSwiglu) {
        const int f = c0 + tx * 4;
        if (f >= F) continue;
        const long long r = static_cast<long long>(off) + m0 + m;
        float act[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) act[j] = swiglu(acc[i][j], acc[i][4 + j]);
        store4(static_cast<T*>(p.out) + r * F + f, act);
        if (p.out2 != nullptr) {
          T* pre = static_cast<T*>(p.out2) + r * p.N;
          store4(pre + f, acc[i]);
          store4(pre + F + f, acc[i] + 4);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = c0 + h * 64 + tx * 4;
          if (c >= cols) continue;
          float* v = acc[i] + h * 4;
          if constexpr (kind == kProdDgradSwiglu) {
            const long long r = (static_cast<long long>(off) + m0 + m) * 2 * p.K;
            float dg[4], du[4];
            if (m0 + m < cnt) {
              float g[4], u[4];
              load4(static_cast<const T*>(p.pre) + r + c, g);
              load4(static_cast<const T*>(p.pre) + r + p.K + c, u);
#pragma unroll
              for (int j = 0; j < 4; ++j) swiglu_bwd(g[j], u[j], v[j], &dg[j], &du[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) dg[j] = du[j] = 0.0f;
            }
            store4(static_cast<T*>(p.out) + r + c, dg);
            store4(static_cast<T*>(p.out) + r + p.K + c, du);
          } else if constexpr (kind == kProdWgrad) {
            const long long at = w0 + (static_cast<long long>(m0) + m) * p.K + c;
            if (p.out_f32) {
              float* o = static_cast<float*>(p.out) + at;
              if (p.accumulate)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += o[j];
              store4(o, v);
            } else {
              T* o = static_cast<T*>(p.out) + at;
              if (p.accumulate) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += to_f32(o[j]);
              }
              store4(o, v);
            }
          } else {
            store4(static_cast<T*>(p.out) + (static_cast<long long>(off) + m0 + m) * cols + c, v);
          }
        }
      }
    }
    __syncthreads();  // the next tile's first store to shared memory
  }
}

template <typename T>
cudaError_t launch_typed(const ProductParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(num_sms * 2), block(kThreads);
  switch (p.kind) {
    case kProdFwd: return launch_pdl(ep_product_simt_kernel<T, kProdFwd>, grid, block, 0, s, 0, p);
    case kProdFwdSwiglu: return launch_pdl(ep_product_simt_kernel<T, kProdFwdSwiglu>, grid, block, 0, s, 0, p);
    case kProdDgrad: return launch_pdl(ep_product_simt_kernel<T, kProdDgrad>, grid, block, 0, s, 0, p);
    case kProdDgradSwiglu: return launch_pdl(ep_product_simt_kernel<T, kProdDgradSwiglu>, grid, block, 0, s, 0, p);
    default: return launch_pdl(ep_product_simt_kernel<T, kProdWgrad>, grid, block, 0, s, 0, p);
  }
}

}  // namespace

cudaError_t launch_product_simt(const ProductParams& p, int num_sms, cudaStream_t s) {
  return launch_typed<float>(p, num_sms, s);
}

}  // namespace ep
