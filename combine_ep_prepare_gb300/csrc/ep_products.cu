// ep_products.cu -- products grouped by expert of float32 rows, on the CUDA
// cores (the tensor cores have no float32 operands).
//
// For every expert e with rows [off_e, off_e + c_e):
//   forward   out[r][n] = sum_k a[r][k] w[e][n][k]
//   dgrad     out[r][k] = sum_n a[r][n] w[e][n][k]
//   wgrad     out[e][n][k] (+)= sum_r a[r][n] b[r][k]
// with the gated activation silu(gate) * up, or its derivative, applied to the
// sums.  Sums are float32 fused multiply-adds in ascending order of the
// reduction.
#include "ep_experts.cuh"

namespace ep {
namespace {

constexpr int kPad = 4;  // shared-memory row padding against bank conflicts

// Output tiles of TILE x TILE, 8 x 8 sums per thread, STEP reduction elements
// at a time: a thread moves eight elements of each operand per step.
template <int TILE>
struct Shape {
  static constexpr int kThreads = (TILE / 8) * (TILE / 8);
  static constexpr int kStep = kThreads * 8 / TILE;
  using Row = float[TILE + kPad];
};

__device__ __forceinline__ void load8(const float* p, float* v) {
  *reinterpret_cast<float4*>(v) = reinterpret_cast<const float4*>(p)[0];
  *reinterpret_cast<float4*>(v + 4) = reinterpret_cast<const float4*>(p)[1];
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Two float32 multiply-adds in one instruction.
__device__ __forceinline__ void fma2(float2* c, const float2& a, const float2& b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;"
      : "+l"(*reinterpret_cast<unsigned long long*>(c))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)), "l"(*reinterpret_cast<const unsigned long long*>(&b)));
}

// One operand's share of a step.  kc: the reduction index is the contiguous one.
template <int TILE, bool kc>
struct Slab {
  static constexpr int kParts = kc ? Shape<TILE>::kStep / 8 : TILE / 8;  // runs of eight in a contiguous row
  float v[8];
  static __device__ __forceinline__ int mn() { return kc ? threadIdx.x / kParts : threadIdx.x % kParts * 8; }
  static __device__ __forceinline__ int k() { return kc ? threadIdx.x % kParts * 8 : threadIdx.x / kParts; }
  // base: element (0, 0); ld: elements between rows; mn / k limits.
  __device__ __forceinline__ void load(const float* base, long long ld, int mn_lim, int k0, int k_lim) {
    const int m = mn(), kk = k0 + k();
    if (m < mn_lim && kk < k_lim) {
      load8(kc ? base + m * ld + kk : base + kk * ld + m, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  }
  __device__ __forceinline__ void store(typename Shape<TILE>::Row* s) const {
    if constexpr (kc) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k() + i][mn()] = v[i];
    } else {
      store4(&s[k()][mn()], v);
      store4(&s[k()][mn() + 4], v + 4);
    }
  }
};

// A tile per block, rows and columns of a thread in two runs of four, TILE / 2
// apart, so that a warp's shared-memory reads of four floats do not collide;
// the next step's loads are in flight while the present one is multiplied.  In
// the gated forward one half of the tile's columns are gate columns and the
// other the up columns of the same features, so that one thread holds both.
// PER_SM: blocks per SM that the registers are to leave room for, 0 as the
// compiler has it.
template <int TILE, int PER_SM, int kind>
__global__ void __launch_bounds__(Shape<TILE>::kThreads, PER_SM) ep_product_simt_kernel(const ProductParams p) {
  constexpr int kThreads = Shape<TILE>::kThreads, kStep = Shape<TILE>::kStep, kTile = TILE, kHalf = TILE / 2;
  constexpr bool rows_out = kind != kProdWgrad;
  constexpr bool a_kc = rows_out;
  constexpr bool b_kc = kind == kProdFwd || kind == kProdFwdSwiglu;
  __shared__ __align__(16) float sa[2][kStep][kTile + kPad];
  __shared__ __align__(16) float sb[2][kStep][kTile + kPad];
  __shared__ int cum[EP_MAX_EXPERTS + 1];
  __shared__ int part[32];
  pdl_wait();
  if (!blocks_ok(p.hdr, p.R)) return;
  const int t = threadIdx.x, tx = t % (TILE / 8), ty = t / (TILE / 8);
  const float* a = static_cast<const float*>(p.a);
  const float* b = static_cast<const float*>(p.b);
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
    const float *ab, *bb;
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
    alignas(8) float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;

    Slab<TILE, a_kc> la;
    Slab<TILE, b_kc> lb;
    auto load = [&](int k0) {
      la.load(ab, ald, a_lim, k0, red);
      if constexpr (kind == kProdFwdSwiglu) {
        // slab columns below kHalf: gate features from c0 on, the others: up features from c0 on
        const int lim = b_lim < kHalf ? b_lim : kHalf;
        const bool up = lb.mn() >= kHalf;
        lb.load(bb + (up ? (static_cast<long long>(F) - kHalf) * bld : 0), bld, up ? kHalf + lim : lim, k0, red);
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
          float ra[8];
          alignas(16) float2 rb[4];
          *reinterpret_cast<float4*>(ra) = *reinterpret_cast<const float4*>(&sa[buf][k][ty * 4]);
          *reinterpret_cast<float4*>(ra + 4) = *reinterpret_cast<const float4*>(&sa[buf][k][kHalf + ty * 4]);
          *reinterpret_cast<float4*>(rb) = *reinterpret_cast<const float4*>(&sb[buf][k][tx * 4]);
          *reinterpret_cast<float4*>(rb + 2) = *reinterpret_cast<const float4*>(&sb[buf][k][kHalf + tx * 4]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) fma2(reinterpret_cast<float2*>(&acc[i][2 * j]), make_float2(ra[i], ra[i]), rb[j]);
        }
        if (more) {
          la.store(sa[buf ^ 1]);
          lb.store(sb[buf ^ 1]);
        }
        __syncthreads();
        buf ^= 1;
      }
    }
    // Epilogue: rows m0 + {0, kHalf} + 4 ty + i.  A padding row's sums are +0
    // (its operand was not read), so it gets zeros without a case of its own,
    // except through the activation's derivative, which reads `pre`.
    const int m_lim = rows_out ? rows - m0 : p.N - m0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = (i >> 2) * kHalf + ty * 4 + (i & 3);
      if (m >= m_lim) continue;
      if constexpr (kind == kProdFwdSwiglu) {
        const int f = c0 + tx * 4;
        if (f >= F) continue;
        const long long r = static_cast<long long>(off) + m0 + m;
        float act[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) act[j] = swiglu(acc[i][j], acc[i][4 + j]);
        store4(static_cast<float*>(p.out) + r * F + f, act);
        if (p.out2 != nullptr) {
          float* pre = static_cast<float*>(p.out2) + r * p.N;
          store4(pre + f, acc[i]);
          store4(pre + F + f, acc[i] + 4);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = c0 + h * kHalf + tx * 4;
          if (c >= cols) continue;
          float* v = acc[i] + h * 4;
          if constexpr (kind == kProdDgradSwiglu) {
            const long long r = (static_cast<long long>(off) + m0 + m) * 2 * p.K;
            float dg[4], du[4];
            if (m0 + m < cnt) {
              const float* g = static_cast<const float*>(p.pre) + r + c;
#pragma unroll
              for (int j = 0; j < 4; ++j) swiglu_bwd(g[j], g[p.K + j], v[j], &dg[j], &du[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) dg[j] = du[j] = 0.0f;
            }
            store4(static_cast<float*>(p.out) + r + c, dg);
            store4(static_cast<float*>(p.out) + r + p.K + c, du);
          } else if constexpr (kind == kProdWgrad) {
            const long long at = w0 + (static_cast<long long>(m0) + m) * p.K + c;
            float* o = static_cast<float*>(p.out) + at;
            if (p.accumulate) {
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] += o[j];
            }
            store4(o, v);
          } else {
            store4(static_cast<float*>(p.out) + (static_cast<long long>(off) + m0 + m) * cols + c, v);
          }
        }
      }
    }
    __syncthreads();  // the next tile's first store to shared memory
  }
}

template <int TILE, int PER_SM>
cudaError_t launch_tile(const ProductParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(2 * num_sms), block(Shape<TILE>::kThreads);
  switch (p.kind) {
    case kProdFwd: return launch_pdl(ep_product_simt_kernel<TILE, PER_SM, kProdFwd>, grid, block, 0, s, 0, p);
    case kProdFwdSwiglu: return launch_pdl(ep_product_simt_kernel<TILE, PER_SM, kProdFwdSwiglu>, grid, block, 0, s, 0, p);
    case kProdDgrad: return launch_pdl(ep_product_simt_kernel<TILE, PER_SM, kProdDgrad>, grid, block, 0, s, 0, p);
    default: return launch_pdl(ep_product_simt_kernel<TILE, PER_SM, kProdDgradSwiglu>, grid, block, 0, s, 0, p);
  }
}

}  // namespace

// Tiles of 128 x 128 read least.  Two blocks per SM hide each other's
// latencies (dgrad of 8 x 1,024 rows x 2 x 1024 -> 2048 1.73 -> 1.42 ms), but
// with hardly a tile per SM the device puts pairs of them on some SMs and none
// on others (2,000 rows x 1024 -> 1024, 160 tiles: 105 -> 193 us), hence one
// where the buffer's capacity of rows makes fewer than three tiles per SM.
// wgrad, whose operands both lie along the tile's sides, takes 64 x 64 tiles:
// 2.94 ms for 3.29 at 16 experts x 512 rows x 4096 x 2048.
cudaError_t launch_product_simt(const ProductParams& p, int num_sms, cudaStream_t s) {
  if (p.kind == kProdWgrad)
    return launch_pdl(ep_product_simt_kernel<64, 8, kProdWgrad>, dim3(8 * num_sms), dim3(Shape<64>::kThreads), 0, s, 0, p);
  const long long cols = p.kind == kProdFwd || p.kind == kProdFwdSwiglu ? p.N : p.K;
  const long long tiles = (p.R / 128 + (p.E < p.R ? p.E : p.R)) * ((cols + 127) / 128);
  return tiles < 3ll * num_sms ? launch_tile<128, 0>(p, num_sms, s) : launch_tile<128, 2>(p, num_sms, s);
}

}  // namespace ep
