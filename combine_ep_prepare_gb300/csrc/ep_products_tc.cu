// ep_products_tc.cu -- products grouped by expert on the tensor cores (bf16
// and fp16), tcgen05.mma with accumulators in tensor memory.
//
// For every expert e with rows [off_e, off_e + c_e):
//   forward   out[r][n] = sum_k a[r][k] w[e][n][k]
//   dgrad     out[r][k] = sum_n a[r][n] w[e][n][k]
//   wgrad     out[e][n][k] (+)= sum_r a[r][n] b[r][k]
// and the gated activation, or its derivative, on the float32 sums.
//
// The features are the M side of the mma and the rows of an expert its N
// side: features are a multiple of a tile in practice, while N may be any
// multiple of 32, so a ragged expert costs little more than its rows and an
// expert with three rows costs its weights' bytes.  An expert's rows are cut
// into even blocks of at most 256.  (In wgrad M is the input features and N
// the output features, so that a warp's stores run along dw's rows.)
//
// A pair of blocks (a cluster of two SMs) shares a tile of 256 features x up
// to 256 rows: each SM holds 128 features' operand and half of the rows, so
// that per 16 reduction steps an SM's shared memory takes 8 KB in and gives
// 8 KB out in the 128 clocks of the mma.  One SM alone on 128 x 256 would
// move 24 KB; on 16,384 rows x 7168 -> 2 x 2048 that version reached 1.22
// PFLOP/s, this one 1.65 with 512 rows to each expert and 1.47 with ragged
// ones.  The pairs are persistent.  In each block two warps move 64-wide slabs
// of the two operands into a ring of stages by TMA; one warp of the first
// block issues the mma for both; eight warps read the finished accumulator and
// write the output while the next tile is multiplied (two accumulators of 256
// columns fill tensor memory).  With large experts the mma bound it: a slab's
// take 590 clocks where the nominal rate gives 512 (750 in wgrad, whose second
// operand is MN-major too); with a few rows to each expert the weights' bytes
// do (6.4 to 6.6 TB/s).  No operand is laid out anew: what is contiguous along
// the reduction is read K-major (rows, and the weights of the forward pass),
// what is not MN-major (the weights of dgrad, both operands of wgrad).
//
// Ragged ends.  A row block may read the rows of the next expert: they fill
// accumulator columns that are not stored.  The features' ends are the tensor
// maps' bounds, which read as zeros.  In wgrad the rows are the reduction:
// the last slab's mma stop at the 16 rows holding the last one, and the rows
// of those 16 beyond it are zeroed in shared memory first, since they may
// hold anything.
#include <algorithm>
#include <atomic>

#include "ep_pack.cuh"
#include "ep_tc.cuh"

namespace ep {
namespace {

constexpr int kEpilogueWarps = 8;  // two for each 32 accumulator lanes
constexpr int kThreads = (4 + kEpilogueWarps) * 32;
constexpr int kTileM = 256, kTileN = 256, kSlab = 64;  // of the pair
constexpr int kHalfM = kTileM / 2;
constexpr int kABytes = kHalfM * kSlab * 2, kBBytes = kTileN / 2 * kSlab * 2;
constexpr int kStages = 6;
constexpr int kBoxBytes = kSlab * 128;  // 64 rows of 64 elements
// The accumulator in tensor memory is rounded toward zero with every mma: a
// weight gradient of 512 rows is off by 4.7e-7 (of its norm), of 4,096 by
// 4.4e-6, of 16,384 by 1.9e-5, all to one side.  That drowns in a 16-bit
// result up to kLong slabs (32,768 elements: 4e-5 beside the 2e-4 of fp16's
// rounding).  Longer sums are taken in parts of kLong slabs: each is added in
// float32, rounded to nearest, to what the other accumulator's columns carry
// of the parts before, so that the error stays there at any length (2^20
// elements in one sum were off by 1.2e-3).  A float32 gradient is summed over
// segments of twelve slabs (768 rows, 7e-7): each is added to the output in
// float32, rounded to nearest, by the lanes that wrote the one before.  Twelve
// is between the cost of the additions and the error, which grows with the
// segment: 2048 x 2048 gradients of 64 experts x 640 rows take 413, 291, 292
// us with 8, 12, 16 slabs, 64 x 1,000 rows 580, 483, 422, 16 x 3,000 rows 430,
// 348, 310, 8 x 8,192 rows 589, 463, 425.
constexpr int kSegment = 12;
constexpr int kLong = 512;
// Whether a tile's sum is taken in parts, and how many slabs each has.
template <typename O>
__device__ __forceinline__ bool folded(int slabs) { return sizeof(O) != 4 && slabs > kLong; }
template <typename O>
__device__ __forceinline__ int part_slabs(int slabs) { return sizeof(O) == 4 ? kSegment : min(slabs, kLong); }

// f0: first feature; r0, n: first row and row count (N, a multiple of 32) of
// the pair's tile (wgrad: output features).
struct Tile {
  int e, f0, r0, n, cnt, off, rows, slabs;
  bool last;
};

__device__ __forceinline__ int row_blocks(int cnt) { return (cnt + kTileN - 1) / kTileN; }

// The walk over tiles, the same in every role: an expert's row blocks one
// after the other on the same features, so that the pairs at work at one time
// share weights in L2.
template <int kind>
struct Walk {
  const ProductParams& p;
  const int* cum;  // row blocks of the experts before e
  long long total;
  int ftiles, ntiles, e;
  __device__ Walk(const ProductParams& p_, const int* cum_) : p(p_), cum(cum_), e(0) {
    constexpr int per = kind == kProdFwdSwiglu ? kTileM / 2 : kTileM;
    const int cols = kind == kProdFwd ? p.N : kind == kProdFwdSwiglu ? p.N / 2 : p.K;
    ftiles = (cols + per - 1) / per;
    ntiles = (p.N + kTileN - 1) / kTileN;  // wgrad
    total = kind == kProdWgrad ? static_cast<long long>(p.E) * ntiles * ftiles
                               : static_cast<long long>(cum[p.E]) * ftiles;
  }
  __device__ __forceinline__ void at(long long t, Tile* o) {
    constexpr int per = kind == kProdFwdSwiglu ? kTileM / 2 : kTileM;
    if constexpr (kind == kProdWgrad) {
      const long long each = static_cast<long long>(ntiles) * ftiles;
      o->e = static_cast<int>(t / each);
      const int in = static_cast<int>(t - o->e * each);
      o->f0 = in % ftiles * per;
      o->r0 = in / ftiles * kTileN;
      o->n = min(kTileN, (p.N - o->r0 + 31) & ~31);
      o->off = p.offsets[o->e];
      o->cnt = p.counts[o->e];
      o->rows = p.N;
      o->last = false;
      o->slabs = (o->cnt + kSlab - 1) / kSlab;
    } else {
      while (t >= static_cast<long long>(cum[e + 1]) * ftiles) ++e;
      const int in = static_cast<int>(t - static_cast<long long>(cum[e]) * ftiles);
      const int nb = cum[e + 1] - cum[e], b = in % nb;
      o->e = e;
      o->f0 = in / nb * per;
      o->off = p.offsets[e];
      o->cnt = p.counts[e];
      o->rows = p.offsets[e + 1] - o->off;
      o->n = ((o->cnt + nb - 1) / nb + 31) & ~31;
      o->r0 = b * o->n;
      o->last = b + 1 == nb;
      if (o->last) o->n = (o->cnt - o->r0 + 31) & ~31;
      o->slabs = ((kind == kProdFwd || kind == kProdFwdSwiglu ? p.K : p.N) + kSlab - 1) / kSlab;
    }
  }
};

// cum[e] = row blocks of the experts before e.
__device__ __forceinline__ void scan_row_blocks(const ProductParams& p, int* cum, int* part) {
  int base = 0;
  for (int e0 = 0; e0 < p.E; e0 += kThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int v = block_scan<kThreads>(e < p.E ? row_blocks(p.counts[e]) : 0, part);
    if (e < p.E) cum[e + 1] = base + v;
    if (threadIdx.x == kThreads - 1) part[0] = v;
    __syncthreads();
    base += part[0];
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[0] = 0;
  __syncthreads();
}

// The four warps of one half of the epilogue.
__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); }

// The same, true when `ok` is in all four.
__device__ __forceinline__ bool half_all(int half, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, %2, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(1 + half)
      : "memory");
  return all != 0;
}

constexpr int kRows = 16;  // tile rows per step of the epilogue

// Half of a tile goes to the output, kRows rows at a time: accumulator lane l
// of a block is feature l of its 128, column j is row j of the tile, so the
// four warps put their 32 features side by side into shared memory and read
// the rows back, four rows and all 128 features a warp.  A store then covers
// whole 128-byte lines of one row.
template <typename T, int kind, typename O>
struct Rows {
  const ProductParams& p;
  const Tile& t;
  int f, cols, stop;  // this lane's first feature; row length; first row not to be stored (0: no row)
  long long at;       // element of feature f in the tile's first row of the output

  __device__ __forceinline__ Rows(const ProductParams& p_, const Tile& t_, int rank, int lane) : p(p_), t(t_) {
    // four features side by side, or two of the 64 that a block has of a gated pair
    f = kind == kProdFwdSwiglu ? t.f0 + rank * (kHalfM / 2) + 2 * lane : t.f0 + rank * kHalfM + 4 * lane;
    const int width = kind == kProdFwd ? p.N : kind == kProdFwdSwiglu ? p.N / 2 : p.K;
    cols = kind == kProdDgradSwiglu ? 2 * p.K : width;
    stop = f < width ? (kind == kProdWgrad ? p.N : t.cnt) - t.r0 : 0;
    const long long row0 = (kind == kProdWgrad ? static_cast<long long>(t.e) * p.N : t.off) + t.r0;
    at = row0 * cols + (f < width ? f : 0);
  }
  __device__ __forceinline__ const uint2* pre(int r, int up) const {
    return reinterpret_cast<const uint2*>(static_cast<const T*>(p.pre) + at + static_cast<long long>(r) * cols + (up ? p.K : 0));
  }
  // Adds what wgrad's output holds.
  __device__ __forceinline__ void add_old(int r, float4* x) const {
    const long long i = at + static_cast<long long>(r) * cols;
    const float4 y = load4(static_cast<const T*>(p.out) + i);
    *x = make_float4(x->x + y.x, x->y + y.y, x->z + y.z, x->w + y.w);
  }
  // Row r of the tile from the sums x (gated: gate and up of two features).
  __device__ __forceinline__ void put(int r, const float4& x, uint2 raw_g, uint2 raw_u) const {
    const long long i = at + static_cast<long long>(r) * cols;
    T* out = static_cast<T*>(p.out) + i;
    if constexpr (kind == kProdFwdSwiglu) {
      store2(out, x.x * fast_sigmoid(x.x) * x.z, x.y * fast_sigmoid(x.y) * x.w);
      if (p.out2 != nullptr) {
        T* q = static_cast<T*>(p.out2) + 2 * i - f;  // rows twice as long
        store2(q, x.x, x.y);
        store2(q + cols, x.z, x.w);
      }
    } else if constexpr (kind == kProdDgradSwiglu) {
      const float4 g = unpack4<T>(raw_g), u = unpack4<T>(raw_u);
      const float s0 = fast_sigmoid(g.x), s1 = fast_sigmoid(g.y), s2 = fast_sigmoid(g.z), s3 = fast_sigmoid(g.w);
      store4(out, make_float4(x.x * u.x * s0 * (1.0f + g.x * (1.0f - s0)), x.y * u.y * s1 * (1.0f + g.y * (1.0f - s1)),
                              x.z * u.z * s2 * (1.0f + g.z * (1.0f - s2)), x.w * u.w * s3 * (1.0f + g.w * (1.0f - s3))));
      store4(out + p.K, make_float4(x.x * g.x * s0, x.y * g.y * s1, x.z * g.z * s2, x.w * g.w * s3));
    } else if constexpr (sizeof(O) == 4) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + i) = x;
    } else {
      store4(out, x);
    }
  }
};

// One part of a long sum: this warp's lanes and columns of the accumulator are
// added to what the carried ones hold (first: they become it).
__device__ __forceinline__ void carry_half(uint32_t acc, uint32_t carried, int half, int n, bool first) {
#pragma unroll 1
  for (int c = kRows * half; c < n; c += 2 * kRows) {
    float v[kRows], old[kRows];
    __syncwarp();
    tc::tmem_ld16(acc + c, v);
    if (!first) tc::tmem_ld16(carried + c, old);
    tc::tmem_ld_wait();
    if (!first) {
#pragma unroll
      for (int j = 0; j < kRows; ++j) v[j] += old[j];
    }
    tc::tmem_st16(carried + c, v);
  }
  tc::tmem_st_wait();
}

template <typename T, int kind, typename O>
__device__ __forceinline__ void write_half(const ProductParams& p, const Tile& t, uint32_t acc, int rank, int w, int half,
                                           int lane, float* stage, bool add) {
  if constexpr (sizeof(O) == 4) {
    // float32 gradients: a lane's feature of one row from 32 lanes is a whole
    // line as it is.
    const int f = t.f0 + rank * kHalfM + w * 32 + lane, stop = f < p.K ? p.N - t.r0 : 0;
    float* out = static_cast<float*>(p.out) + (static_cast<long long>(t.e) * p.N + t.r0) * p.K + f;
#pragma unroll 1
    for (int c = 32 * half; c < t.n; c += 64) {
      float v[32];
      __syncwarp();
      tc::tmem_ld32(acc + c, v);
      tc::tmem_ld_wait();
      float* o = out + static_cast<long long>(c) * p.K;
      if (c + 32 <= stop) {
        if (add) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += o[static_cast<long long>(j) * p.K];
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) __stcs(o + static_cast<long long>(j) * p.K, v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + j < stop) o[static_cast<long long>(j) * p.K] = add ? v[j] + o[static_cast<long long>(j) * p.K] : v[j];
      }
    }
    return;
  }
  const Rows<T, kind, O> rows(p, t, rank, lane);
  constexpr bool gated = kind == kProdFwdSwiglu || kind == kProdDgradSwiglu;
  // What needs no arithmetic after the sum is rounded before it is put: a
  // word holds two rows' values of a feature, and shared memory, which the
  // tensor core reads its operands from meanwhile, moves half the bytes.
  constexpr bool packed = !gated;
  uint2 raw[2][4] = {};  // dgrad through the activation: gate and up values, read a step ahead of their use
  auto load_pre = [&](int r0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i < rows.stop) {
        raw[0][i] = __ldg(rows.pre(r0 + i, 0));
        raw[1][i] = __ldg(rows.pre(r0 + i, 1));
      }
  };
  if constexpr (kind == kProdDgradSwiglu) load_pre(kRows * half + 4 * w);
  float* put = stage + w * 32 + lane;
  const float* get = stage + (packed ? 2 : 4) * w * kHalfM + (kind == kProdFwdSwiglu ? (lane >> 3) * 32 + 2 * (lane & 7) : 4 * lane);
#pragma unroll 1
  for (int c = kRows * half; c < t.n; c += 2 * kRows) {
    float v[kRows];
    __syncwarp();
    tc::tmem_ld16(acc + c, v);
    tc::tmem_ld_wait();
    const int r0 = c + 4 * w;
    if (kind == kProdWgrad && add) {
      // The old values are added in float32, before the rounding: the rows
      // go through shared memory unrounded, eight at a time.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 8; ++j) put[j * kHalfM] = v[8 * h + j];
        half_sync(half);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float4 x = *reinterpret_cast<const float4*>(stage + (2 * w + i) * kHalfM + 4 * lane);
          const int r = c + 8 * h + 2 * w + i;
          if (r < rows.stop) {
            rows.add_old(r, &x);
            rows.put(r, x, raw[0][0], raw[1][0]);
          }
        }
        half_sync(half);
      }
      continue;
    }
    if constexpr (packed) {
#pragma unroll
      for (int j = 0; j < kRows; j += 2) put[j / 2 * kHalfM] = __uint_as_float(pack2<T>(v[j], v[j + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < kRows; ++j) put[j * kHalfM] = v[j];
    }
    half_sync(half);
    if constexpr (packed) {
      uint2 y[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 q = *reinterpret_cast<const uint4*>(get + i * kHalfM);
        y[2 * i] = make_uint2(__byte_perm(q.x, q.y, 0x5410), __byte_perm(q.z, q.w, 0x5410));
        y[2 * i + 1] = make_uint2(__byte_perm(q.x, q.y, 0x7632), __byte_perm(q.z, q.w, 0x7632));
      }
      half_sync(half);  // read: the next rows may be put
      T* out = static_cast<T*>(p.out) + rows.at + static_cast<long long>(r0) * rows.cols;
      if (r0 + 3 < rows.stop) {
#pragma unroll
        for (int i = 0; i < 4; ++i) __stcs(reinterpret_cast<uint2*>(out + static_cast<long long>(i) * rows.cols), y[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i < rows.stop) *reinterpret_cast<uint2*>(out + static_cast<long long>(i) * rows.cols) = y[i];
      }
    } else {
      float4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kind == kProdFwdSwiglu) {
          // gate features 16 q + m sit at 32 q + m, their up rows 16 further on
          const float2 g = *reinterpret_cast<const float2*>(get + i * kHalfM);
          const float2 u = *reinterpret_cast<const float2*>(get + i * kHalfM + 16);
          x[i] = make_float4(g.x, g.y, u.x, u.y);
        } else {
          x[i] = *reinterpret_cast<const float4*>(get + i * kHalfM);
        }
      }
      half_sync(half);
      if (r0 + 3 < rows.stop) {
#pragma unroll
        for (int i = 0; i < 4; ++i) rows.put(r0 + i, x[i], raw[0][i], raw[1][i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i < rows.stop) rows.put(r0 + i, x[i], raw[0][i], raw[1][i]);
      }
      if constexpr (kind == kProdDgradSwiglu) load_pre(r0 + 2 * kRows);
    }
  }
}

// Rows [begin, end) of the tile (counted from its first) become zeros.
template <typename T, int kind, typename O>
__device__ __forceinline__ void zero_rows(const ProductParams& p, const Tile& t, int rank, int lane, int begin, int end) {
  const Rows<T, kind, O> rows(p, t, rank, lane);
  if (rows.stop == 0) return;
  // A zero gate and a zero sum make every output zero.
  for (int r = begin; r < end; r += kEpilogueWarps)
    rows.put(r, make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_uint2(0, 0), make_uint2(0, 0));
}

// A wait of the whole warp: true when every lane's was.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, gave_up));
}

struct Shared {
  uint64_t full[kStages];      // first block's: both blocks' operands are in
  uint64_t landed[kStages];    // wgrad: this block's ragged slab is in
  uint64_t empty[kStages], acc_full[2], acc_empty[2], drained;
  uint32_t tmem;
  int gave_up, ok;
  int part[32];
  int cum[EP_MAX_EXPERTS + 1];
};
constexpr size_t kSmemBytes =
    static_cast<size_t>(kStages) * (kABytes + kBBytes) + 2 * kRows * kHalfM * sizeof(float) + 1024 + sizeof(Shared);

template <typename T, int kind, typename O>
__global__ void __launch_bounds__(kThreads, 1)
    ep_product_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ CUtensorMap map_b64, const __grid_constant__ CUtensorMap map_b32,
                         const __grid_constant__ CUtensorMap map_b16, const ProductParams p) {
  constexpr bool a_mn = kind == kProdWgrad || kind == kProdDgrad || kind == kProdDgradSwiglu;
  constexpr bool b_mn = kind == kProdWgrad;
  extern __shared__ unsigned char raw[];
  // Aligned by an offset, so that accesses stay known as shared-memory ones.
  unsigned char* ring = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  float* rows_out = reinterpret_cast<float*>(ring + static_cast<size_t>(kStages) * (kABytes + kBBytes));
  Shared& s = *reinterpret_cast<Shared*>(rows_out + 2 * kRows * kHalfM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(tc::cluster_rank());
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map_a);
    tc::tma_prefetch_desc(&map_b);
    tc::tma_prefetch_desc(&map_b16);
    for (int i = 0; i < kStages; ++i) {
      // The first block's two loaders account for both blocks' copies.  A
      // ragged slab of wgrad lands in each block by itself, and each block's
      // zeroing warp then arrives.
      tc::mbar_init(tc::smem_addr(&s.full[i]), 2);
      tc::mbar_init(tc::smem_addr(&s.landed[i]), 2);
      tc::mbar_init(tc::smem_addr(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_addr(&s.acc_full[i]), 1);
      tc::mbar_init(tc::smem_addr(&s.acc_empty[i]), 2 * kEpilogueWarps);
    }
    tc::mbar_init(tc::smem_addr(&s.drained), 1);
    tc::mbar_init_fence();
    s.gave_up = 0;
  }
  if (warp == 2) tc::tmem_alloc(tc::smem_addr(&s.tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = s.tmem;
  pdl_wait();
  if (threadIdx.x == 0) s.ok = blocks_ok(p.hdr, p.R);
  __syncthreads();
  const bool ok = s.ok;
  if (ok && kind != kProdWgrad) scan_row_blocks(p, s.cum, s.part);
  if (ok) {
    Walk<kind> walk(p, s.cum);
    Tile t;
    volatile int* gave_up = &s.gave_up;
    const long long first = blockIdx.x / 2, step = gridDim.x / 2;
    if (warp == 0 || warp == 2) {
      // One warp brings in the features' operand, another the rows': a thread
      // needs 250 to 300 clocks for a copy.  That is why a slab's rows are one
      // copy of 16, 32, 64 or 128 rows, although up to half of them are not
      // this tile's.
      if (lane == 0) {
        const bool load_a = warp == 0;
        int stage = 0;
        uint32_t phase = 0;
        for (long long i = first; i < walk.total && !*gave_up; i += step) {
          walk.at(i, &t);
          const int half = t.n / 2;  // this block's rows
          const int bytes = load_a ? kABytes : b_mn ? (half + 63) / 64 * kBoxBytes : (half > 64 ? 128 : half > 32 ? 64 : half > 16 ? 32 : 16) * 128;
          for (int k = 0; k < t.slabs; ++k) {
            if (!tc::mbar_wait(tc::smem_addr(&s.empty[stage]), phase ^ 1, gave_up)) break;
            const uint32_t a = tc::smem_addr(ring + static_cast<size_t>(stage) * (kABytes + kBBytes)), b = a + kABytes;
            uint32_t bar = rank == 0 ? tc::smem_addr(&s.full[stage]) : tc::in_block(tc::smem_addr(&s.full[stage]), 0);
            if (kind == kProdWgrad && (t.cnt - k * kSlab) < kSlab && ((t.cnt - k * kSlab) & 15)) {
              bar = tc::smem_addr(&s.landed[stage]);  // its rows past the end are zeroed before `full`
              tc::mbar_expect(bar, bytes);
            } else if (rank == 0) {
              tc::mbar_expect(bar, 2 * bytes);  // the other block's copies too
            }
            const int x = k * kSlab;
            if (load_a) {
              if constexpr (kind == kProdWgrad) {
                for (int j = 0; j < kHalfM / 64; ++j)
                  tc::tma_pair_2d(a + j * kBoxBytes, &map_a, bar, t.f0 + rank * kHalfM + j * 64, t.off + x);
              } else if constexpr (kind == kProdFwd) {
                tc::tma_pair_3d(a, &map_a, bar, x, t.f0 + rank * kHalfM, t.e);
              } else if constexpr (kind == kProdFwdSwiglu) {
                for (int j = 0; j < 4; ++j)  // 16 gate rows, then the up rows of the same features
                  tc::tma_pair_4d(a + j * (kABytes / 4), &map_a, bar, x, t.f0 + rank * (kHalfM / 2) + j * 16, 0, t.e);
              } else {
                for (int j = 0; j < kHalfM / 64; ++j)
                  tc::tma_pair_3d(a + j * kBoxBytes, &map_a, bar, t.f0 + rank * kHalfM + j * 64, x, t.e);
              }
            } else if constexpr (kind == kProdWgrad) {
              for (int j = 0; j < (half + 63) / 64; ++j)
                tc::tma_pair_2d(b + j * kBoxBytes, &map_b, bar, t.r0 + rank * half + j * 64, t.off + x);
            } else {
              tc::tma_pair_2d(b, half > 64 ? &map_b : half > 32 ? &map_b64 : half > 16 ? &map_b32 : &map_b16, bar, x,
                              t.off + t.r0 + rank * half);
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        if (load_a) pdl_trigger();
        // Every stage is read out before the block ends.
        for (int j = 0; j < kStages && !*gave_up; ++j) {
          if (!tc::mbar_wait(tc::smem_addr(&s.empty[stage]), phase ^ 1, gave_up)) break;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        // After a wait that gave up, the copies in flight land before the
        // block's shared memory goes; a copy takes microseconds.
        if (*gave_up) {
          const unsigned long long start = tc::now_ns();
          while (tc::now_ns() - start < tc::kWaitNs / 100) {
          }
        }
      }
    } else if (warp == 1 && rank == 0) {
      if (lane == 0) {
        int stage = 0, buf = 0;
        uint32_t phase = 0, acc_phases = 0;  // a bit for each accumulator
        bool lost = false;
        for (long long i = first; i < walk.total && !lost; i += step) {
          walk.at(i, &t);
          if (t.slabs == 0) continue;
          const uint32_t desc = tc::mma_desc(std::is_same<T, __nv_bfloat16>::value, a_mn, b_mn, kTileM, t.n);
          const int segment = part_slabs<O>(t.slabs);
          for (int k0 = 0; k0 < t.slabs && !lost; k0 += segment) {
            lost = !tc::mbar_wait(tc::smem_addr(&s.acc_empty[buf]), (acc_phases >> buf & 1) ^ 1, gave_up);
            if (lost) break;
            tc::fence_after();
            const uint32_t d = tmem + buf * kTileN;
            const int k1 = min(t.slabs, k0 + segment);
            for (int k = k0; k < k1; ++k) {
              const int left = kind == kProdWgrad ? t.cnt - k * kSlab : kSlab;
              // A slab with zeroed rows was handed over by threads of both blocks.
              lost = left < kSlab && (left & 15) ? !tc::mbar_wait<true>(tc::smem_addr(&s.full[stage]), phase, gave_up)
                                                 : !tc::mbar_wait(tc::smem_addr(&s.full[stage]), phase, gave_up);
              if (lost) break;
              tc::fence_after();
              const uint32_t a = tc::smem_addr(ring + static_cast<size_t>(stage) * (kABytes + kBBytes)), b = a + kABytes;
              const uint64_t da = a_mn ? tc::desc_mn_major(a, kBoxBytes) : tc::desc_k_major(a);
              const uint64_t db = b_mn ? tc::desc_mn_major(b, kBoxBytes) : tc::desc_k_major(b);
#pragma unroll
              for (int q = 0; q < kSlab / 16; ++q)
                if (q * 16 < left)
                  tc::mma_f16(d, da + q * (a_mn ? tc::kDescStepMn : tc::kDescStepK),
                              db + q * (b_mn ? tc::kDescStepMn : tc::kDescStepK), desc, k > k0 || q > 0);
              tc::mma_commit(tc::smem_addr(&s.empty[stage]));
              if (k + 1 == k1) tc::mma_commit(tc::smem_addr(&s.acc_full[buf]));
              if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
              }
            }
            acc_phases ^= 1u << buf;
            // A sum in parts keeps to one accumulator, the tile after it too:
            // the other one carries the sum until this one is released last.
            if (!folded<O>(t.slabs)) buf ^= 1;
          }
        }
        if (lost) {
          // What was issued ends before tensor memory is freed.
          tc::mma_commit(tc::smem_addr(&s.drained));
          const unsigned long long start = tc::now_ns();
          while (!tc::mbar_try(tc::smem_addr(&s.drained), 0) && tc::now_ns() - start < tc::kWaitNs) {
          }
        }
      }
    } else if (warp == 3 && kind == kProdWgrad) {
      // Ragged slabs: rows left .. 16 ceil(left / 16) - 1 become zeros.
      int stage = 0;
      uint32_t phases = 0;
      for (long long i = first; i < walk.total; i += step) {
        walk.at(i, &t);
        const int left = t.cnt & (kSlab - 1);
        stage = (stage + t.slabs) % kStages;
        if ((left & 15) == 0) continue;
        const int at = (stage + kStages - 1) % kStages;
        if (!warp_wait(tc::smem_addr(&s.landed[at]), (phases >> at) & 1, gave_up)) break;
        phases ^= 1u << at;
        unsigned char* slab = ring + static_cast<size_t>(at) * (kABytes + kBBytes);
        const int chunks = (16 - (left & 15)) * 8, boxes = kHalfM / 64 + (t.n / 2 + 63) / 64;
        for (int j = lane; j < chunks * boxes; j += 32)
          *reinterpret_cast<uint4*>(slab + j / chunks * kBoxBytes + left * 128 + j % chunks * 16) = make_uint4(0, 0, 0, 0);
        // Each lane's fence orders its zeros before the asynchronous proxy's
        // reads; the arrival hands them to the thread that issues the mma, in
        // the second block with a release for the cluster.  (That release and
        // its acquire cost 71 us of 483 at 128 experts x 500 rows, where every
        // tile has such a slab: 512 rows take 412.)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) tc::mbar_arrive(tc::smem_addr(&s.full[at]));
          else tc::mbar_publish_cluster(tc::in_block(tc::smem_addr(&s.full[at]), 0));
        }
      }
    } else if (warp >= 4) {
      int buf = 0;
      uint32_t acc_phases = 0;
      const int half = (warp - 4) >> 2;
      const int w = warp & 3;  // the accumulator lanes a warp can reach go by its number
      for (long long i = first; i < walk.total; i += step) {
        walk.at(i, &t);
        const bool has = t.slabs > 0;
        if (!has && p.accumulate) continue;  // an expert without rows keeps its gradient
        auto wait = [&]() {
          // The four warps go on or leave together: write_half has barriers.
          const bool ok = half_all(half, tc::mbar_wait(tc::smem_addr(&s.acc_full[buf]), acc_phases >> buf & 1, gave_up));
          tc::fence_after();
          return ok;
        };
        auto release = [&]() {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_cluster(tc::in_block(tc::smem_addr(&s.acc_empty[buf]), 0));
          acc_phases ^= 1u << buf;
          if (!folded<O>(t.slabs)) buf ^= 1;
        };
        const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
        bool fine = true;
        const int segment = part_slabs<O>(t.slabs);
        for (int k = 0; k < t.slabs && fine; k += segment) {
          fine = wait();
          if (!fine) break;
          uint32_t acc = tmem + buf * kTileN + lanes;
          if (folded<O>(t.slabs)) {
            const uint32_t carried = tmem + (buf ^ 1) * kTileN + lanes;
            carry_half(acc, carried, half, t.n, k == 0);
            acc = carried;
          }
          if (!folded<O>(t.slabs) || k + segment >= t.slabs)
            write_half<T, kind, O>(p, t, acc, rank, w, half, lane, rows_out + half * kRows * kHalfM,
                                   p.accumulate || (sizeof(O) == 4 && k > 0));
          release();
        }
        if (!fine) break;
        // Padding rows; wgrad: the gradient of an expert without rows.
        if (kind == kProdWgrad ? !has : t.last)
          zero_rows<T, kind, O>(p, t, rank, lane, (kind == kProdWgrad ? 0 : t.cnt - t.r0) + warp - 4,
                             kind == kProdWgrad ? min(t.n, p.N - t.r0) : t.rows - t.r0);
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && s.gave_up) atomicOr(&p.hdr[kHdrStatus], static_cast<int>(EP_ST_TIMEOUT));
  tc::cluster_sync();  // neither block leaves while the other may reach into it
  tc::fence_after();
  if (warp == 2) tc::tmem_free(tmem, 512);
}

// A map of [dim 3]..[dim 1][dim 0] two-byte elements, strides in elements.
bool make_map(CUtensorMap* m, const void* base, int dtype, int dims, const long long (&size)[4],
              const long long (&stride)[3], const int (&box)[4]) {
  const tc::EncodeFn f = tc::tensor_map_encoder();
  if (f == nullptr) return false;
  cuuint64_t sz[4], st[3];
  cuuint32_t bx[4];
  const cuuint32_t one[4] = {1, 1, 1, 1};
  for (int i = 0; i < dims; ++i) {
    sz[i] = static_cast<cuuint64_t>(size[i]);
    bx[i] = static_cast<cuuint32_t>(box[i]);
    if (i + 1 < dims) st[i] = static_cast<cuuint64_t>(stride[i]) * 2;
  }
  return f(m, dtype == EP_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
           static_cast<cuuint32_t>(dims), const_cast<void*>(base), sz, st, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [R][cols] in boxes of 64 columns; weights [E][N][K] likewise.
bool rows_map(CUtensorMap* m, const void* base, int dtype, long long cols, long long rows, int box_rows) {
  return make_map(m, base, dtype, 2, {cols, rows, 1, 1}, {cols, 0, 0}, {kSlab, box_rows, 1, 1});
}
bool weights_map(CUtensorMap* m, const ProductParams& p, int box_rows) {
  const long long K = p.K, N = p.N;
  return make_map(m, p.b, p.dtype, 3, {K, N, p.E, 1}, {K, N * K, 0}, {kSlab, box_rows, 1, 1});
}
// Gate and up halves: [E][2][F][K], boxes of 16 rows of each.
bool gated_map(CUtensorMap* m, const ProductParams& p) {
  const long long K = p.K, F = p.N / 2;
  return make_map(m, p.b, p.dtype, 4, {K, F, 2, p.E}, {K, F * K, 2 * F * K}, {kSlab, 16, 2, 1});
}

// Pairs of blocks that fit on the current device at once (0: the query
// failed); the kernel's shared memory is raised on the way.  Once per device.
template <typename T, int kind, typename O>
int resident_pairs(int num_sms) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int pairs = known[dev].load(std::memory_order_acquire);
  if (pairs == 0) {
    const auto kern = ep_product_tc_kernel<T, kind, O>;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes)) != cudaSuccess)
      return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms / 2 * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg) != cudaSuccess || pairs < 1) return 0;
    pairs = std::min(pairs, num_sms / 2);
    known[dev].store(pairs, std::memory_order_release);
  }
  return pairs;
}

template <typename T, int kind, typename O = T>
cudaError_t launch_kind(const ProductParams& p, int num_sms, cudaStream_t s) {
  CUtensorMap a, b, b64, b32, b16;
  const long long R = p.R > 0 ? p.R : 1;  // without rows nothing is read through the maps
  bool ok;
  if (kind == kProdWgrad) {
    ok = rows_map(&a, p.b, p.dtype, p.K, R, kSlab) && rows_map(&b, p.a, p.dtype, p.N, R, kSlab);
    b64 = b32 = b16 = b;  // not used
  } else {
    const bool fwd = kind == kProdFwd || kind == kProdFwdSwiglu;
    ok = (kind == kProdFwdSwiglu ? gated_map(&a, p) : weights_map(&a, p, fwd ? kHalfM : kSlab)) &&
         rows_map(&b, p.a, p.dtype, fwd ? p.K : p.N, R, 128) && rows_map(&b64, p.a, p.dtype, fwd ? p.K : p.N, R, 64) &&
         rows_map(&b32, p.a, p.dtype, fwd ? p.K : p.N, R, 32) && rows_map(&b16, p.a, p.dtype, fwd ? p.K : p.N, R, 16);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int pairs = resident_pairs<T, kind, O>(num_sms);
  if (pairs == 0) return cudaErrorLaunchOutOfResources;
  return launch_pdl(ep_product_tc_kernel<T, kind, O>, dim3(2 * pairs), dim3(kThreads), kSmemBytes, s, 2, a, b, b64, b32, b16, p);
}

template <typename T>
cudaError_t launch_typed(const ProductParams& p, int num_sms, cudaStream_t s) {
  switch (p.kind) {
    case kProdFwd: return launch_kind<T, kProdFwd>(p, num_sms, s);
    case kProdFwdSwiglu: return launch_kind<T, kProdFwdSwiglu>(p, num_sms, s);
    case kProdDgrad: return launch_kind<T, kProdDgrad>(p, num_sms, s);
    case kProdDgradSwiglu: return launch_kind<T, kProdDgradSwiglu>(p, num_sms, s);
    default: return p.out_f32 ? launch_kind<T, kProdWgrad, float>(p, num_sms, s) : launch_kind<T, kProdWgrad>(p, num_sms, s);
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
