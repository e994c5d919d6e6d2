// ep_products.cu -- products grouped by expert of float32 rows, on the CUDA
// cores (the tensor cores have no float32 operands).
//
// For every expert e with rows [off_e, off_e + c_e):
//   forward   out[r][n] = sum_k a[r][k] w[e][n][k]
//   dgrad     out[r][k] = sum_n a[r][n] w[e][n][k]
//   wgrad     out[e][n][k] (+)= sum_r a[r][n] b[r][k]
// with the gated activation silu(gate) * up, or its derivative, applied to the
// sums.  Sums are float32 fused multiply-adds, two chains in ascending order of
// the reduction (elements 0 to 7 and 8 to 15 of every 16) added at the end; in
// tiles of eight rows or fewer, a chain per lane or thread and a tree.
#include "ep_experts.cuh"

namespace ep {
namespace {

// Output tiles of 64 x 64, 8 x 8 sums per thread, 16 reduction elements at a
// time, of which each of two groups of 64 threads multiplies eight.  What
// bounds the kernel is the shared memory's reads, four of 16 bytes for the 64
// multiply-adds of a thread and reduction element, 81% busy while the
// multiply-add unit is 63% (8 experts x 1,024 rows, 1024 -> 2048: 786 us for a
// floor of 430 at the CUDA cores' 80 TFLOP/s; 8,192 rows x 2048 -> 2 x 1024
// take 1.59 ms).  The weight gradient, whose operands are written to shared
// memory as they lie, takes 666 us there (71% and 68%).  Larger tiles save no
// such reads.  128 x 128 by one group of 256 threads took the same there, but
// leaves SMs without work where tiles are few (2,500 rows of 8 experts, 1024
// -> 1024: 206 us for 137; 800 rows of 4: 106 for 63) and multiplies more
// padding where experts have few rows (64 experts x 25 rows: 365 for 216).
// 16 x 8 sums per thread read a quarter less and leave two warps per
// scheduler, too few for the loads' latency (1.72 ms).
constexpr int kTile = 64, kHalf = kTile / 2;
constexpr int kGroup = (kTile / 8) * (kTile / 8), kThreads = 2 * kGroup;
constexpr int kStep = 16;
constexpr int kPerSm = 4;  // blocks that the registers leave room for
constexpr int kPad = 4;    // shared-memory row padding against bank conflicts
static_assert(kTile * kStep == 8 * kThreads, "a thread moves eight elements of each operand per step");

__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Two float32 multiply-adds in one instruction.
__device__ __forceinline__ void fma2(float2* c, const float2& a, const float2& b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;"
      : "+l"(*reinterpret_cast<unsigned long long*>(c))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)), "l"(*reinterpret_cast<const unsigned long long*>(&b)));
}

// One operand's share of a step: two runs of four elements, half of a
// contiguous row apart, so that the lanes of a warp write to different banks.
// kc: the reduction index is the contiguous one.
template <bool kc>
struct Slab {
  static constexpr int kRow = kc ? kStep : kTile;
  static constexpr int kParts = kRow / 8;
  alignas(16) float v[2][4];
  static __device__ __forceinline__ int at(int c) { return c * (kRow / 2) + threadIdx.x % kParts * 4; }
  static __device__ __forceinline__ int row() { return threadIdx.x / kParts; }
  // base: element (0, 0); ld: elements between rows; mn / k limits.
  __device__ __forceinline__ void load(const float* base, long long ld, int mn_lim, int k0, int k_lim) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int m = kc ? row() : at(c), k = k0 + (kc ? at(c) : row());
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (m < mn_lim && k < k_lim) x = *reinterpret_cast<const float4*>(kc ? base + m * ld + k : base + k * ld + m);
      *reinterpret_cast<float4*>(v[c]) = x;
    }
  }
  __device__ __forceinline__ void store(float (*s)[kTile + kPad]) const {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if constexpr (kc) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[at(c) + i][row()] = v[c][i];
      } else {
        store4(&s[row()][at(c)], v[c]);
      }
    }
  }
};

// Tiles of a few rows are bound by the weights' bytes: their blocks read the
// weights as they lie, straight into registers, and keep no operand in shared
// memory.  Warps wait for those loads three quarters of their time: one row
// each of 32 experts, 1024 -> 4096, takes 111 us, 4.9 TB/s, for a floor of 79.
// 16 tokens' top 2 of 32 experts, 1024 -> 4096: 139 us for 333 by the way of
// full tiles; one token's top 2 of 8, 1024 -> 1024: 12.5 for 38.  Eight rows by
// four columns are the sums that a thread has registers for beside the loads.
// wgrad is not treated so: sums straight from global memory gained 11% with two
// rows to each expert and cost 2% with 512.  Sums go to part[..][row][column].
constexpr int kThin = 8;
using Thin = float[kThin][kTile];

// Four columns at a time per warp, the lanes along the reduction.  column(c):
// the weights of the tile's column c, or nullptr.
template <class Column>
__device__ __forceinline__ void thin_along(const float* a, long long ald, int rows, int red, Column column, Thin& part) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int c = warp * (kTile / 4); c < (warp + 1) * (kTile / 4); c += 4) {
    const float* w = column(c);
    if (w == nullptr) continue;
    const long long ld = column(c + 1) - w;
    float s[4 * kThin];  // [column][row]
#pragma unroll
    for (int i = 0; i < 4 * kThin; ++i) s[i] = 0.0f;
#pragma unroll 1
    for (int k = lane * 4; k < red; k += 128) {
      float4 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(w + j * ld + k);
#pragma unroll
      for (int r = 0; r < kThin; ++r) {
        if (r < rows) {
          const float4 x = *reinterpret_cast<const float4*>(a + r * ald + k);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[j * kThin + r] = fmaf(x.w, b[j].w, fmaf(x.z, b[j].z, fmaf(x.y, b[j].y, fmaf(x.x, b[j].x, s[j * kThin + r]))));
        }
      }
    }
    // Lanes trade halves of what they hold until lane i has the whole sum i.
#pragma unroll
    for (int h = 2 * kThin; h > 0; h /= 2) {
#pragma unroll
      for (int i = 0; i < h; ++i) {
        const float keep = lane & h ? s[i + h] : s[i], give = lane & h ? s[i] : s[i + h];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
      }
    }
    part[lane % kThin][c + lane / kThin] = s[0];
  }
}

// Four columns per thread, eight threads of each four along the reduction,
// four elements at a time; the sums of a warp's two are added here.
__device__ __forceinline__ void thin_across(const float* a, long long ald, int rows, const float* b, long long bld, int cols, int red,
                                            Thin* part) {
  const int lane = threadIdx.x % 32, c = threadIdx.x % 16 * 4;
  float s[kThin][4];
#pragma unroll
  for (int r = 0; r < kThin; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[r][j] = 0.0f;
  if (c < cols) {
#pragma unroll 1
    for (int k = threadIdx.x / 16 * 4; k < red; k += kThreads / 4) {
      float4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(b + (k + i) * bld + c);
#pragma unroll
      for (int r = 0; r < kThin; ++r) {
        if (r < rows) {
          const float4 x = *reinterpret_cast<const float4*>(a + r * ald + k);
          s[r][0] = fmaf(x.w, w[3].x, fmaf(x.z, w[2].x, fmaf(x.y, w[1].x, fmaf(x.x, w[0].x, s[r][0]))));
          s[r][1] = fmaf(x.w, w[3].y, fmaf(x.z, w[2].y, fmaf(x.y, w[1].y, fmaf(x.x, w[0].y, s[r][1]))));
          s[r][2] = fmaf(x.w, w[3].z, fmaf(x.z, w[2].z, fmaf(x.y, w[1].z, fmaf(x.x, w[0].z, s[r][2]))));
          s[r][3] = fmaf(x.w, w[3].w, fmaf(x.z, w[2].w, fmaf(x.y, w[1].w, fmaf(x.x, w[0].w, s[r][3]))));
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kThin; ++r) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[r][j] += __shfl_xor_sync(0xffffffffu, s[r][j], 16);
    if (lane < 16) store4(&part[threadIdx.x / 32][r][c], s[r]);
  }
}

// A tile per block, rows and columns of a thread in two runs of four, kHalf
// apart, so that a warp's shared-memory reads of four floats do not collide;
// the next step's loads are in flight while the present one is multiplied.  In
// the gated forward one half of the tile's columns are gate columns and the
// other the up columns of the same features, so that one thread holds both.
template <int kind>
__global__ void __launch_bounds__(kThreads, kPerSm) ep_product_simt_kernel(const ProductParams p) {
  constexpr bool rows_out = kind != kProdWgrad;
  constexpr bool a_kc = rows_out;
  constexpr bool b_kc = kind == kProdFwd || kind == kProdFwdSwiglu;
  __shared__ __align__(16) float sa[2][kStep][kTile + kPad];
  __shared__ __align__(16) float sb[2][kStep][kTile + kPad];
  __shared__ int cum[EP_MAX_EXPERTS + 1];
  __shared__ int part[32];
  pdl_wait();
  if (!blocks_ok(p.hdr, p.R)) return;
  const int group = threadIdx.x / kGroup, t = threadIdx.x % kGroup, tx = t % (kTile / 8), ty = t / (kTile / 8);
  const float* a = static_cast<const float*>(p.a);
  const float* b = static_cast<const float*>(p.b);
  const int F = p.N / 2;
  constexpr int cols_per_tile = kind == kProdFwdSwiglu ? kHalf : kTile;
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
    const bool thin = rows_out && a_lim > 0 && a_lim <= kThin;
    constexpr int parts = b_kc ? 1 : kThreads / 32;
    static_assert(sizeof(sa) >= parts * sizeof(Thin), "the parts have room");
    Thin* part = reinterpret_cast<Thin*>(&sa[0][0][0]);
    if (thin) {
      if constexpr (b_kc) {
        thin_along(ab, ald, a_lim, red, [&](int c) -> const float* {
          const bool up = kind == kProdFwdSwiglu && c >= kHalf;
          const int in = up ? c - kHalf : c;
          if (in >= (kind == kProdFwdSwiglu && b_lim > kHalf ? kHalf : b_lim)) return nullptr;
          return bb + (static_cast<long long>(in) + (up ? F : 0)) * bld;
        }, part[0]);
      } else {
        thin_across(ab, ald, a_lim, bb, bld, b_lim, red, part);
      }
      __syncthreads();
    }
    alignas(16) float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;

    Slab<a_kc> la;
    Slab<b_kc> lb;
    auto load = [&](int k0) {
      la.load(ab, ald, a_lim, k0, red);
      if constexpr (kind == kProdFwdSwiglu) {
        // slab columns below kHalf: gate features from c0 on, the others: up features from c0 on
        const int lim = b_lim < kHalf ? b_lim : kHalf;
        const bool up = lb.row() >= kHalf;
        lb.load(bb + (up ? (static_cast<long long>(F) - kHalf) * bld : 0), bld, up ? kHalf + lim : lim, k0, red);
      } else {
        lb.load(bb, bld, b_lim, k0, red);
      }
    };
    if (thin) {
      if (group == 0 && ty * 4 < a_lim) {
        for (int w = 0; w < parts; ++w) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] += part[w][ty * 4 + i][(j >> 2) * kHalf + tx * 4 + (j & 3)];
        }
      }
    } else if (a_lim > 0 && red > 0) {
      load(0);
      la.store(sa[0]);
      lb.store(sb[0]);
      __syncthreads();
      int buf = 0;
      for (int k0 = 0; k0 < red; k0 += kStep) {
        const bool more = k0 + kStep < red;
        if (more) load(k0 + kStep);
#pragma unroll 2
        for (int ki = 0; ki < kStep / 2; ++ki) {
          const int k = group * (kStep / 2) + ki;
          alignas(16) float ra[8];
          alignas(16) float2 rb[4];
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            *reinterpret_cast<float4*>(ra + i) = *reinterpret_cast<const float4*>(&sa[buf][k][i / 4 * kHalf + ty * 4]);
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
    // The groups' sums are added, group 0's first: group 0 finishes the rows of
    // i < 4 (in acc[0..3]), group 1 the others.
    static_assert(sizeof(sa) >= kGroup * 32 * sizeof(float), "half of a group's sums have room");
    float4* sums = reinterpret_cast<float4*>(&sa[0][0][0]);
    if (!thin) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (group != g) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sums[i * kGroup + t] = reinterpret_cast<float4*>(acc[g * 4])[i];
        }
        __syncthreads();
        if (group == g) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 o = sums[i * kGroup + t];
            const float* mine = &acc[g * 4 + (i >> 1)][(i & 1) * 4];
            float* v = &acc[i >> 1][(i & 1) * 4];
            v[0] = mine[0] + o.x, v[1] = mine[1] + o.y, v[2] = mine[2] + o.z, v[3] = mine[3] + o.w;
          }
        }
        __syncthreads();
      }
    }
    // Epilogue: rows m0 + kHalf group + 4 ty + i.  A padding row's operand was
    // not read but taken as zero, which an infinite weight makes NaN: its sums
    // are set to zero.
    const int m_lim = rows_out ? rows - m0 : p.N - m0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = group * kHalf + ty * 4 + i;
      if (m >= m_lim) continue;
      if (rows_out && m0 + m >= cnt) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
      }
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

}  // namespace

cudaError_t launch_product_simt(const ProductParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(kPerSm * num_sms), block(kThreads);
  switch (p.kind) {
    case kProdFwd: return launch_pdl(ep_product_simt_kernel<kProdFwd>, grid, block, 0, s, 0, p);
    case kProdFwdSwiglu: return launch_pdl(ep_product_simt_kernel<kProdFwdSwiglu>, grid, block, 0, s, 0, p);
    case kProdDgrad: return launch_pdl(ep_product_simt_kernel<kProdDgrad>, grid, block, 0, s, 0, p);
    case kProdDgradSwiglu: return launch_pdl(ep_product_simt_kernel<kProdDgradSwiglu>, grid, block, 0, s, 0, p);
    default: return launch_pdl(ep_product_simt_kernel<kProdWgrad>, grid, block, 0, s, 0, p);
  }
}

}  // namespace ep
