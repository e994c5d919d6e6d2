// ep_products_tc.cu -- products grouped by expert on the tensor cores (bf16
// and fp16), tcgen05.mma with accumulators in tensor memory.
//
// For every expert e with rows [off_e, off_e + c_e):
//   forward   out[r][n] = sum_k a[r][k] w[e][n][k]
//   dgrad     out[r][k] = sum_n a[r][n] w[e][n][k]
//   wgrad     out[e][n][k] (+)= sum_r a[r][n] b[r][k]
// and the gated activation, or its derivative, on the float32 sums.
//
// A persistent block per SM walks output tiles of 128 x 256.  One warp moves
// 64-wide slabs of both operands into a ring of shared-memory stages by TMA,
// one issues the mma, four read finished accumulators and write the output
// while the next tile is multiplied (two accumulators of 256 columns fill the
// SM's tensor memory).  No operand is laid out anew: what is contiguous along
// the reduction is read as a K-major operand (rows, and the weights of the
// forward pass), what is not as an MN-major one (the weights of dgrad, both
// operands of wgrad).
//
// Ragged ends.  Row tiles start at each expert's first row, so a tile may
// read the rows of the next expert: they fill accumulator rows that are not
// stored.  The features' ends are the tensor maps' bounds, which read as
// zeros.  In wgrad the rows are the reduction: the last slab's mma stop at
// the 16 rows holding the last one, and the rows of those 16 beyond it are
// zeroed in shared memory first, since they may hold anything.
#include <algorithm>
#include <atomic>

#include "ep_experts.cuh"
#include "ep_tc.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kTileM = 128, kTileN = 256, kSlab = 64;
constexpr int kABytes = kTileM * kSlab * 2, kBBytes = kTileN * kSlab * 2;
constexpr int kStages = 4;
constexpr int kBlockBytes = kSlab * 128;  // 64 reduction rows of 64 elements

struct Tile {
  int e, m0, c0, off, cnt, rows, slabs;
};

// The walk over tiles, the same in every role: row blocks of a column block
// one after the other, so that the blocks at work at one time share weights.
template <int kind>
struct Walk {
  const ProductParams& p;
  const int* cum;
  long long total;
  int ntiles, mtiles, e;
  __device__ Walk(const ProductParams& p_, const int* cum_) : p(p_), cum(cum_), e(0) {
    constexpr int per = kind == kProdFwdSwiglu ? kTileN / 2 : kTileN;
    const int cols = kind == kProdFwd ? p.N : kind == kProdFwdSwiglu ? p.N / 2 : p.K;
    ntiles = (cols + per - 1) / per;
    mtiles = (p.N + kTileM - 1) / kTileM;  // wgrad
    total = kind == kProdWgrad ? static_cast<long long>(p.E) * ntiles * mtiles
                               : static_cast<long long>(cum[p.E]) * ntiles;
  }
  __device__ __forceinline__ void at(long long t, Tile* o) {
    constexpr int per = kind == kProdFwdSwiglu ? kTileN / 2 : kTileN;
    if constexpr (kind == kProdWgrad) {
      const long long each = static_cast<long long>(ntiles) * mtiles;
      o->e = static_cast<int>(t / each);
      const int in = static_cast<int>(t - o->e * each);
      o->m0 = in % mtiles * kTileM;
      o->c0 = in / mtiles * per;
      o->off = p.offsets[o->e];
      o->cnt = p.counts[o->e];
      o->rows = p.N;
      o->slabs = (o->cnt + kSlab - 1) / kSlab;
    } else {
      while (t >= static_cast<long long>(cum[e + 1]) * ntiles) ++e;
      const int in = static_cast<int>(t - static_cast<long long>(cum[e]) * ntiles);
      const int mt = cum[e + 1] - cum[e];
      o->e = e;
      o->m0 = in % mt * kTileM;
      o->c0 = in / mt * per;
      o->off = p.offsets[e];
      o->cnt = p.counts[e];
      o->rows = p.offsets[e + 1] - o->off;
      const int red = kind == kProdFwd || kind == kProdFwdSwiglu ? p.K : p.N;
      o->slabs = o->m0 < o->cnt ? (red + kSlab - 1) / kSlab : 0;
    }
  }
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Eight values rounded to T in one 16-byte store.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<T>(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// One accumulator row of a tile, `acc` its tensor-memory address (lane and
// first column), m the row in the tile; has: the tile was multiplied.
template <typename T, int kind>
__device__ __forceinline__ void write_row(const ProductParams& p, const Tile& t, uint32_t acc, int m, bool has) {
  const int row = t.m0 + m;
  if constexpr (kind == kProdFwdSwiglu) {
    const int F = p.N / 2;
    const long long r = static_cast<long long>(t.off) + row;
    T* act = static_cast<T*>(p.out) + r * F + t.c0;
    T* pre = p.out2 == nullptr ? nullptr : static_cast<T*>(p.out2) + r * p.N + t.c0;
#pragma unroll 1
    for (int c = 0; c < kTileN / 2; c += 16) {
      if (t.c0 + c >= F) break;
      float g[16], u[16];
      __syncwarp();
      if (has) {
        tc::tmem_ld16(acc + c, g);
        tc::tmem_ld16(acc + kTileN / 2 + c, u);
        tc::tmem_ld_wait();
      }
      if (row >= t.cnt) {
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = u[i] = 0.0f;
      }
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        if (t.c0 + c + h >= F || row >= t.rows) break;
        if (pre != nullptr) {
          store8(pre + c + h, g + h);
          store8(pre + F + c + h, u + h);
        }
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = swiglu(g[h + i], u[h + i]);
        store8(act + c + h, a);
      }
    }
  } else if constexpr (kind == kProdDgradSwiglu) {
    const long long r = (static_cast<long long>(t.off) + row) * 2 * p.K + t.c0;
#pragma unroll 1
    for (int c = 0; c < kTileN; c += 16) {
      if (t.c0 + c >= p.K) break;
      float v[16];
      __syncwarp();
      if (has) {
        tc::tmem_ld16(acc + c, v);
        tc::tmem_ld_wait();
      }
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        if (t.c0 + c + h >= p.K || row >= t.rows) break;
        float dg[8], du[8];
        if (row < t.cnt) {
          float g[8], u[8];
          load8(static_cast<const T*>(p.pre) + r + c + h, g);
          load8(static_cast<const T*>(p.pre) + r + p.K + c + h, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) swiglu_bwd(g[i], u[i], v[h + i], &dg[i], &du[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dg[i] = du[i] = 0.0f;
        }
        store8(static_cast<T*>(p.out) + r + c + h, dg);
        store8(static_cast<T*>(p.out) + r + p.K + c + h, du);
      }
    }
  } else {
    const int cols = kind == kProdFwd ? p.N : p.K;
    const long long r = kind == kProdWgrad ? static_cast<long long>(t.e) * p.N + row : static_cast<long long>(t.off) + row;
    const long long at = r * cols + t.c0;
#pragma unroll 1
    for (int c = 0; c < kTileN; c += 32) {
      if (t.c0 + c >= cols) break;
      float v[32];
      __syncwarp();
      if (has) {
        tc::tmem_ld32(acc + c, v);
        tc::tmem_ld_wait();
      }
      if (kind == kProdWgrad ? !has : row >= t.cnt) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
      }
#pragma unroll
      for (int h = 0; h < 32; h += 8) {
        if (t.c0 + c + h >= cols || row >= t.rows) break;
        if (kind == kProdWgrad && p.out_f32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at + c + h);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float4 x = make_float4(v[h + 4 * q], v[h + 4 * q + 1], v[h + 4 * q + 2], v[h + 4 * q + 3]);
            if (p.accumulate) {
              const float4 y = o[q];
              x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            o[q] = x;
          }
        } else {
          T* o = static_cast<T*>(p.out) + at + c + h;
          if (kind == kProdWgrad && p.accumulate) {
            float y[8];
            load8(o, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[h + i] += y[i];
          }
          store8(o, v + h);
        }
      }
    }
  }
}

// A wait of the whole warp: true when every lane's was.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, gave_up));
}

struct Shared {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
  uint32_t tmem;
  int gave_up, ok;
  int part[32];
  int cum[EP_MAX_EXPERTS + 1];
};
constexpr size_t kSmemBytes = static_cast<size_t>(kStages) * (kABytes + kBBytes) + 1024 + sizeof(Shared);

template <typename T, int kind>
__global__ void __launch_bounds__(kThreads, 1)
    ep_product_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const ProductParams p) {
  constexpr bool a_mn = kind == kProdWgrad;
  constexpr bool b_mn = kind == kProdWgrad || kind == kProdDgrad || kind == kProdDgradSwiglu;
  extern __shared__ unsigned char raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  Shared& s = *reinterpret_cast<Shared*>(ring + static_cast<size_t>(kStages) * (kABytes + kBBytes));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map_a);
    tc::tma_prefetch_desc(&map_b);
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(tc::smem_addr(&s.full[i]), 1);
      tc::mbar_init(tc::smem_addr(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_addr(&s.acc_full[i]), 1);
      tc::mbar_init(tc::smem_addr(&s.acc_empty[i]), 4);
    }
    tc::mbar_init(tc::smem_addr(&s.drained), 1);
    tc::mbar_init_fence();
    s.gave_up = 0;
  }
  if (warp == 2) tc::tmem_alloc(tc::smem_addr(&s.tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s.tmem;
  pdl_wait();
  if (threadIdx.x == 0) s.ok = blocks_ok(p.hdr, p.R);
  __syncthreads();
  const bool ok = s.ok;
  if (ok && kind != kProdWgrad) scan_row_tiles<kThreads>(p.offsets, p.E, kTileM, s.cum, s.part);
  if (ok) {
    Walk<kind> walk(p, s.cum);
    Tile t;
    volatile int* gave_up = &s.gave_up;
    if (warp == 0) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        for (long long i = blockIdx.x; i < walk.total && !*gave_up; i += gridDim.x) {
          walk.at(i, &t);
          for (int k = 0; k < t.slabs; ++k) {
            if (!tc::mbar_wait(tc::smem_addr(&s.empty[stage]), phase ^ 1, gave_up)) break;
            const uint32_t full = tc::smem_addr(&s.full[stage]);
            const uint32_t a = tc::smem_addr(ring + static_cast<size_t>(stage) * (kABytes + kBBytes)), b = a + kABytes;
            tc::mbar_expect(full, kABytes + kBBytes);
            const int x = k * kSlab;
            if constexpr (kind == kProdWgrad) {
              for (int j = 0; j < kTileM / 64; ++j)
                tc::tma_load_2d(a + j * kBlockBytes, &map_a, full, t.m0 + j * 64, t.off + x);
              for (int j = 0; j < kTileN / 64; ++j)
                tc::tma_load_2d(b + j * kBlockBytes, &map_b, full, t.c0 + j * 64, t.off + x);
            } else {
              tc::tma_load_2d(a, &map_a, full, x, t.off + t.m0);
              if constexpr (b_mn) {
                for (int j = 0; j < kTileN / 64; ++j)
                  tc::tma_load_3d(b + j * kBlockBytes, &map_b, full, t.c0 + j * 64, x, t.e);
              } else if constexpr (kind == kProdFwdSwiglu) {
                tc::tma_load_3d(b, &map_b, full, x, t.c0, t.e);
                tc::tma_load_3d(b + kBBytes / 2, &map_b, full, x, p.N / 2 + t.c0, t.e);
              } else {
                tc::tma_load_3d(b, &map_b, full, x, t.c0, t.e);
              }
            }
            ++issued;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        if (!*gave_up) {
          // Every stage is read out before the block ends.
          for (int j = 0; j < kStages; ++j) {
            if (!tc::mbar_wait(tc::smem_addr(&s.empty[stage]), phase ^ 1, gave_up)) break;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        } else {
          // The copies in flight land before the block's shared memory goes.
          const int n = static_cast<int>(issued < kStages ? issued : kStages);
          const unsigned long long start = tc::now_ns();
          for (int j = 0; j < n; ++j) {
            if (--stage < 0) {
              stage = kStages - 1;
              phase ^= 1;
            }
            while (!tc::mbar_try(tc::smem_addr(&s.full[stage]), phase) && tc::now_ns() - start < tc::kWaitNs) {
            }
          }
        }
      }
    } else if (warp == 1) {
      constexpr uint32_t desc = tc::mma_desc(sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value, a_mn, b_mn, kTileM, kTileN);
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (long long i = blockIdx.x; i < walk.total; i += gridDim.x) {
        walk.at(i, &t);
        if (t.slabs == 0) continue;
        if (!warp_wait(tc::smem_addr(&s.acc_empty[buf]), acc_phase ^ 1, gave_up)) break;
        tc::fence_after();
        const uint32_t d = tmem + buf * kTileN;
        bool lost = false;
        for (int k = 0; k < t.slabs; ++k) {
          if (!warp_wait(tc::smem_addr(&s.full[stage]), phase, gave_up)) {
            lost = true;
            break;
          }
          tc::fence_after();
          unsigned char* slab = ring + static_cast<size_t>(stage) * (kABytes + kBBytes);
          int steps = kSlab / 16;
          if constexpr (kind == kProdWgrad) {
            const int left = t.cnt - k * kSlab;
            if (left < kSlab) {
              steps = (left + 15) / 16;
              // Rows left .. 16 steps - 1 of each 64-element block: zeros.
              const int chunks = (16 * steps - left) * 8;
              for (int j = lane; j < chunks * ((kTileM + kTileN) / 64); j += 32)
                *reinterpret_cast<uint4*>(slab + j / chunks * kBlockBytes + left * 128 + j % chunks * 16) =
                    make_uint4(0, 0, 0, 0);
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
            }
          }
          if (lane == 0) {
            const uint32_t a = tc::smem_addr(slab), b = a + kABytes;
            const uint64_t da = a_mn ? tc::desc_mn_major(a, kBlockBytes) : tc::desc_k_major(a);
            const uint64_t db = b_mn ? tc::desc_mn_major(b, kBlockBytes) : tc::desc_k_major(b);
#pragma unroll
            for (int q = 0; q < kSlab / 16; ++q)
              if (q < steps)
                tc::mma_f16(d, da + q * (a_mn ? tc::kDescStepMn : tc::kDescStepK),
                            db + q * (b_mn ? tc::kDescStepMn : tc::kDescStepK), desc, k > 0 || q > 0);
            tc::mma_commit(tc::smem_addr(&s.empty[stage]));
            if (k + 1 == t.slabs) tc::mma_commit(tc::smem_addr(&s.acc_full[buf]));
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (lost) {
          // What was issued ends before tensor memory is freed.
          if (lane == 0) {
            tc::mma_commit(tc::smem_addr(&s.drained));
            const unsigned long long start = tc::now_ns();
            while (!tc::mbar_try(tc::smem_addr(&s.drained), 0) && tc::now_ns() - start < tc::kWaitNs) {
            }
          }
          __syncwarp();
          break;
        }
        if (++buf == 2) {
          buf = 0;
          acc_phase ^= 1;
        }
      }
    } else if (warp >= 4) {
      int buf = 0;
      uint32_t acc_phase = 0;
      const int w = warp - 4;
      for (long long i = blockIdx.x; i < walk.total; i += gridDim.x) {
        walk.at(i, &t);
        const bool has = t.slabs > 0;
        if (has) {
          if (!warp_wait(tc::smem_addr(&s.acc_full[buf]), acc_phase, gave_up)) break;
          tc::fence_after();
        } else if (kind == kProdWgrad && p.accumulate) {
          continue;  // an expert without rows keeps its gradient
        }
        write_row<T, kind>(p, t, tmem + buf * kTileN + (static_cast<uint32_t>(w * 32) << 16), w * 32 + lane, has);
        if (has) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(tc::smem_addr(&s.acc_empty[buf]));
          if (++buf == 2) {
            buf = 0;
            acc_phase ^= 1;
          }
        }
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x == 0 && s.gave_up) atomicOr(&p.hdr[kHdrStatus], static_cast<int>(EP_ST_TIMEOUT));
  if (warp == 2) tc::tmem_free(tmem, 512);
}

// A map of [depth][rows][cols] two-byte elements read in boxes of 64 columns.
bool make_map(CUtensorMap* m, const void* base, int dtype, int dims, long long cols, long long rows, long long depth,
              int box_rows) {
  const tc::EncodeFn f = tc::tensor_map_encoder();
  if (f == nullptr) return false;
  const cuuint64_t size[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(depth)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(cols) * rows * 2};
  const cuuint32_t box[3] = {kSlab, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return f(m, dtype == EP_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
           static_cast<cuuint32_t>(dims), const_cast<void*>(base), size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int kind>
cudaError_t launch_kind(const ProductParams& p, int num_sms, cudaStream_t s) {
  CUtensorMap a, b;
  const long long R = p.R > 0 ? p.R : 1;  // without rows nothing is read through the maps
  bool ok;
  if (kind == kProdWgrad) {
    ok = make_map(&a, p.a, p.dtype, 2, p.N, R, 1, kSlab) && make_map(&b, p.b, p.dtype, 2, p.K, R, 1, kSlab);
  } else if (kind == kProdDgrad || kind == kProdDgradSwiglu) {
    ok = make_map(&a, p.a, p.dtype, 2, p.N, R, 1, kTileM) && make_map(&b, p.b, p.dtype, 3, p.K, p.N, p.E, kSlab);
  } else {
    ok = make_map(&a, p.a, p.dtype, 2, p.K, R, 1, kTileM) &&
         make_map(&b, p.b, p.dtype, 3, p.K, p.N, p.E, kind == kProdFwdSwiglu ? kTileN / 2 : kTileN);
  }
  if (!ok) return cudaErrorInvalidValue;
  const void* kern = reinterpret_cast<const void*>(ep_product_tc_kernel<T, kind>);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(ep_product_tc_kernel<T, kind>, dim3(num_sms), dim3(kThreads), kSmemBytes, s, 0, a, b, p);
}

template <typename T>
cudaError_t launch_typed(const ProductParams& p, int num_sms, cudaStream_t s) {
  switch (p.kind) {
    case kProdFwd: return launch_kind<T, kProdFwd>(p, num_sms, s);
    case kProdFwdSwiglu: return launch_kind<T, kProdFwdSwiglu>(p, num_sms, s);
    case kProdDgrad: return launch_kind<T, kProdDgrad>(p, num_sms, s);
    case kProdDgradSwiglu: return launch_kind<T, kProdDgradSwiglu>(p, num_sms, s);
    default: return launch_kind<T, kProdWgrad>(p, num_sms, s);
  }
}

}  // namespace

namespace tc {

EncodeFn tensor_map_encoder() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    void* sym = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<EncodeFn>(sym);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

}  // namespace tc

cudaError_t launch_product_tc(const ProductParams& p, int num_sms, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP16) return launch_typed<__half>(p, num_sms, s);
  return launch_typed<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace ep
