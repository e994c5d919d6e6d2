// ep_products_f8.cu -- products grouped by expert of e4m3 rows and weights
// with a scale for each block of 128, on tcgen05.mma.
//
//   forward  out[r][n] = sum_b as[r][b] ws[n/128][b] sum_{k in b} a[r][k] w[n][k]
//   dgrad    out[r][k] = sum_b as[r][b] ws[b][k/128] sum_{n in b} a[r][n] w[n][k]
//
// Tiles are as for the 16-bit products: a pair of SMs takes 256 features (the
// M side, 128 in each SM) times up to 256 rows of an expert (the N side), and
// a slab of the reduction is 128 bytes wide -- here 128 elements, one block of
// the scales.  The scales are arbitrary float32 numbers, so the tensor core
// can sum over one block only: each slab goes to an accumulator in tensor
// memory of its own (two of 256 columns in turn, up to eight where tiles have
// few rows), and eight warps add it to sums in registers, times the row's scale
// and the weights', while the next slab is multiplied into another.
//
// Adding a slab takes a warp 64 packed multiply-adds, 16 loads from tensor
// memory and 8 of the scales.  The loads are 16 lanes x 256 bits, which give a
// lane two columns (rows of the tile) in eight, so that it needs 32 rows'
// scales and not all 128 of its half: with one lane per feature the scales'
// loads alone would keep shared memory busy for 256 clocks a slab, next to the
// operands'.  A warp of its own brings the scales in, four slabs at a time.
//
// With many rows the adding warps bound it, by their latencies: two for each
// scheduler, which wait, load and multiply in turn, while no unit is busy for more
// than 38% of the time.  8 experts x 1,024 rows, 7168 -> 4096,
// take 230 us (2.09 PFLOP/s), 139 without the additions and 221 with one mma of
// four; the additions with neither loads nor mma take 152.  With ragged experts
// (16,384 rows over 32 of them, 7168 -> 2 x 2048, 8-bit result) 557 us, with even
// ones 496; the 16-bit product takes 655 to 712.  With a few rows per expert the
// weights' bytes do: 64 experts x 4 rows, 301 us, 6.2 TB/s; 2048 -> 7168, 145 us,
// 6.5 TB/s.  What it took: sums that stay in their registers (a branch on the
// tile's width in the loop made 115 moves a slab and warp: 889 us for the 496),
// packed multiply-adds from the compiler's own pairs (530), and mma issued from
// uniform registers (up decode 375 us before, 301 after).  Columns per load,
// loads further ahead, stages and the split of registers made no difference; more
// adding warps with fewer sums each were not tried.  The kernels spill 40 to 48
// bytes.  Plain input gradient: 16,384 even rows, 2 x 2048 -> 7168, 484 us
// (1.99 PFLOP/s), 65,536 ragged ones of 128 experts, 2 x 1024 -> 2048, 343; 64
// experts x 4 rows, 270.  (All are times of calls in a row, every expert with
// rows.)
//
// The gated pair: 16 gate rows and the 16 up rows of the same features
// alternate in the tile, and land in one lane's two halves of the sums.  Its
// 8-bit result needs the largest magnitude of a row's 128 features, 64 in each
// SM of the pair: they exchange theirs through distributed shared memory (19 us
// of the 496 beside a 16-bit result).  The two 16-bit results that a backward pass
// reads take 48 us more (545).
#include <algorithm>
#include <atomic>

#include "ep_f8.cuh"
#include "ep_pack.cuh"
#include "ep_tc.cuh"

namespace ep {
namespace {

constexpr int kEpilogueWarps = 8;  // two for each 32 accumulator lanes
constexpr int kThreads = (4 + kEpilogueWarps) * 32;
constexpr int kTileM = 256, kTileN = 256, kSlab = 128;  // of the pair
constexpr int kHalfM = kTileM / 2, kHalfN = kTileN / 2;
constexpr int kABytes = kHalfM * kSlab, kBBytes = kHalfN * kSlab;
// The ring: stages of the features' 16 KB and of the rows' as many bytes as the
// largest tile needs, so that more are in flight where there are few rows.
constexpr int kRingBytes = 6 * (kABytes + kBBytes), kMaxStages = 10;
__device__ __forceinline__ int box_rows(int half) { return half > 64 ? 128 : half > 32 ? 64 : half > 16 ? 32 : 16; }
constexpr int kGroup = 4, kGroups = 2;  // slabs whose scales come together; groups in flight
constexpr int kSlots = 8, kSlotColumns = 512 / kSlots;  // of tensor memory; an accumulator takes 1, 2 or 4
// Registers of a loading warp and of an adding one: 128 threads of the first
// and 256 of the second have what 384 x 168 gave them.
constexpr int kFewRegs = 72, kManyRegs = 216;
static_assert(128 * kFewRegs + 256 * kManyRegs <= kThreads * 168, "more registers than the block is launched with");
// Staging of one half of the epilogue, in words: 16 pairs of rows x 128
// features, or eight pairs in float32.  The paddings keep the lanes of a
// store on different banks.
constexpr int kPairStride = kHalfM + 8, kPairStride32 = kHalfM + 4, kGatedStride = kHalfM / 2 + 8;
constexpr int kStageWords = 16 * kPairStride;
static_assert(8 * 2 * kPairStride32 <= kStageWords && 16 * kGatedStride <= kStageWords, "staging");

struct Tile {
  int e, f0, r0, n, cnt, off, rows;
  bool last;
};

__device__ __forceinline__ int row_blocks(int cnt) { return (cnt + kTileN - 1) / kTileN; }

// The walk over tiles, the same in every role: an expert's row blocks one
// after the other on the same features.
template <int kind>
struct Walk {
  static constexpr int kPer = kind == kProdFwdSwiglu ? kTileM / 2 : kTileM;
  const F8Params& p;
  const int* cum;  // row blocks of the experts before e
  long long total;
  int ftiles, e;
  __device__ Walk(const F8Params& p_, const int* cum_) : p(p_), cum(cum_), e(0) {
    const int cols = kind == kProdFwd ? p.N : kind == kProdFwdSwiglu ? p.N / 2 : p.K;
    ftiles = (cols + kPer - 1) / kPer;
    total = static_cast<long long>(cum[p.E]) * ftiles;
  }
  __device__ __forceinline__ void at(long long t, Tile* o) {
    while (t >= static_cast<long long>(cum[e + 1]) * ftiles) ++e;
    const int in = static_cast<int>(t - static_cast<long long>(cum[e]) * ftiles);
    const int nb = cum[e + 1] - cum[e], b = in % nb;
    o->e = e;
    o->f0 = in / nb * kPer;
    o->off = p.offsets[e];
    o->cnt = p.counts[e];
    o->rows = p.offsets[e + 1] - o->off;
    o->n = ((o->cnt + nb - 1) / nb + 31) & ~31;
    o->r0 = b * o->n;
    o->last = b + 1 == nb;
    if (o->last) o->n = (o->cnt - o->r0 + 31) & ~31;
  }
};

// cum[e] = row blocks of the experts before e; *most (0 before) the rows of the largest expert.
__device__ __forceinline__ void scan_row_blocks(const F8Params& p, int* cum, int* part, int* most) {
  int base = 0;
  for (int e0 = 0; e0 < p.E; e0 += kThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int cnt = e < p.E ? p.counts[e] : 0;
    if (cnt > 0) atomicMax(most, cnt);
    const int v = block_scan<kThreads>(row_blocks(cnt), part);
    if (e < p.E) cum[e + 1] = base + v;
    if (threadIdx.x == kThreads - 1) part[0] = v;
    __syncthreads();
    base += part[0];
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[0] = 0;
  __syncthreads();
}

// The accumulators in tensor memory: tiles of few rows have up to eight in
// turn, which covers the way from an mma's end over the adding warps and back.
// Where the width changes the walk begins again at the first one.
struct Slots {
  int width, at;
  uint32_t phases;  // a bit for each slot's barriers
  __device__ __forceinline__ Slots() : width(0), at(0), phases(0) {}
  static __device__ __forceinline__ int of(int n) { return n > 2 * kSlotColumns ? 4 : n > kSlotColumns ? 2 : 1; }
  __device__ __forceinline__ uint32_t phase() const { return phases >> at & 1; }
  __device__ __forceinline__ void next() {
    phases ^= 1u << at;
    at = (at + width) & (kSlots - 1);
  }
};

// Buffers of the pair's exchange of largest magnitudes, taken by tiles in turn,
// each with barriers of its own.  The other block may publish tile i + 1 when one
// thread of this one has seen tile i; it publishes tile i + 2 only after this
// block's half has published i + 1, all of its threads being past tile i's wait
// by then.  So a barrier for every other tile is never two phases ahead of a
// thread that waits on it, and its buffer is never written while it is read.
constexpr int kExchanges = 2;

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[kSlots], acc_empty[kSlots], drained;
  uint64_t scales_full[kGroups], scales_empty[kGroups], peer_full[kExchanges][2];  // peer_full: of each half
  uint32_t tmem;
  int gave_up, ok, most;  // most: rows of the largest tile
  int part[32];
  float ws[kGroups][2][kGroup];  // weight scales: the features', or gate's and up's
  alignas(16) float peer_max[kExchanges][kTileN];  // the other block's largest magnitudes
  alignas(16) float as[kGroups][kGroup][kTileN];
  int cum[EP_MAX_EXPERTS + 1];
};
constexpr size_t kSmemBytes = static_cast<size_t>(kRingBytes) + 2 * kStageWords * 4 + 1024 + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// A wait of the whole warp: true when every lane's was.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, gave_up));
}

__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); }

// 16 lanes x 16 columns of the accumulator: word 4 i + j of a lane is row
// lane / 4 + 8 (j / 2), column 8 i + 2 (lane % 4) + j % 2.
__device__ __forceinline__ void tmem_ld_rows(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}

// Waits for the loads so far; what is computed from these words stays behind it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[2][8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0][0]), "+r"(r[0][1]), "+r"(r[0][2]), "+r"(r[0][3]), "+r"(r[0][4]), "+r"(r[0][5]), "+r"(r[0][6]), "+r"(r[0][7]),
                 "+r"(r[1][0]), "+r"(r[1][1]), "+r"(r[1][2]), "+r"(r[1][3]), "+r"(r[1][4]), "+r"(r[1][5]), "+r"(r[1][6]), "+r"(r[1][7]));
}

__host__ __device__ constexpr uint32_t mma_desc_f8(bool a_mn, int m, int n) {  // e4m3 operands, float32 sums
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// MN-major e4m3: a row of 128 features per element of the reduction; 32
// elements, one mma's share, are 4096 bytes.
constexpr uint64_t kDescStepMn8 = 4096 >> 4;

// A slab's four mma into accumulator d, and what arrives after them: `empty`
// for the stage, `full` for the accumulator, in both blocks.  The whole warp
// calls it and one lane issues: outside a divergent branch the compiler keeps
// descriptors and addresses in uniform registers, where the instructions want
// them.  (From one lane's branch the issuing thread took 890 clocks a slab.)
template <uint64_t a_step>
__device__ __forceinline__ void mma_slab(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t empty, uint32_t full) {
  asm volatile(
      "{\n .reg .pred e, no, yes;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " setp.ne.u32 no, 0, 0;\n setp.eq.u32 yes, 0, 0;\n"
      " add.u64 a1, %1, %6;\n add.u64 a2, a1, %6;\n add.u64 a3, a2, %6;\n"
      " add.u64 b1, %2, %7;\n add.u64 b2, b1, %7;\n add.u64 b3, b2, %7;\n"
      " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, no;\n"
      " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a1, b1, %3, yes;\n"
      " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a2, b2, %3, yes;\n"
      " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a3, b3, %3, yes;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%4], %8;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], %8;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"(empty), "r"(full), "n"(a_step), "n"(tc::kDescStepK), "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ bool elect() {
  uint32_t is;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}\n" : "=r"(is));
  return is != 0;
}

__device__ __forceinline__ void prefetch_2d(const CUtensorMap* m, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(m), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void store_peer(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A warp's sums of a tile: columns 32 i + 8 j + 2 (lane % 4) + {0, 1} of its
// half's, features lane / 4 + {0, 8} of the first (h = 0) and second 16 of its
// 32 (the gated pair: gate and up of the same features).
struct Sums {
  float2 v[4][2][8];  // [i][h][2 j + (feature >= 8)]
};

// Where the adding warps are in the rings.
struct Turn {
  Slots slots;
  int slot = 0;  // of the scales
  uint32_t phase = 0;
};

// Of a tile's slabs, what an adding warp has of the one at hand.
struct Slab {
  uint32_t acc;     // its part of the accumulator
  const float* as;  // the rows' scales from this lane's first on
  float w0, w1;     // gated: the weights' scales
  float4 x;         // the rows' scales of the 16 columns to come
};

// A tile's slabs, one after the other: 16 times `chunks` columns of the
// accumulator times the scales, to the sums.  While sixteen columns are added
// the next ones and their scales are loaded; when all are in registers the
// accumulator is handed back.  (With the width known here there is no branch
// between loads and sums, and the sums keep their registers.)
//
// A wait that gave up leaves its warp in step with the others, with nothing of
// use in its sums: every later wait ends at once.
template <int kind, int chunks>
struct Adder {
  Sums& a;
  Shared& s;
  Turn& turn;
  uint32_t tmem, empty;  // empty: the first block's barriers of the accumulators
  int lane, slabs, first_column;
  Slab now;
  uint32_t r[2][2][8];

  // Slab k's accumulator is there: its first columns are on their way to r[0].
  __device__ __forceinline__ void begin(int k) {
    volatile int* gave_up = &s.gave_up;
    const int in = k & (kGroup - 1);
    if (in == 0) tc::mbar_wait(tc::smem_addr(&s.scales_full[turn.slot]), turn.phase, gave_up);
    if constexpr (kind == kProdFwdSwiglu) {
      now.w0 = s.ws[turn.slot][0][in];
      now.w1 = s.ws[turn.slot][1][in];
    }
    now.as = &s.as[turn.slot][in][first_column + 4 * (lane & 3)];
    now.x = *reinterpret_cast<const float4*>(now.as);
    tc::mbar_wait(tc::smem_addr(&s.acc_full[turn.slots.at]), turn.slots.phase(), gave_up);
    __syncwarp();
    tc::fence_after();
    now.acc = tmem + turn.slots.at * kSlotColumns;
    load(0);
  }
  __device__ __forceinline__ void load(int c) {
    tmem_ld_rows(now.acc + 16 * c, r[c & 1][0]);
    tmem_ld_rows(now.acc + 16 * c + (16u << 16), r[c & 1][1]);
  }
  // Slab k's accumulator and, with its last slab, the scales' slot are read.
  __device__ __forceinline__ void end(int k) {
    tc::fence_before();
    __syncwarp();
    const bool ends = (k & (kGroup - 1)) == kGroup - 1 || k + 1 == slabs;
    if (lane == 0) {
      tc::mbar_arrive_cluster(empty + 8 * turn.slots.at);
      if (ends) tc::mbar_arrive(tc::smem_addr(&s.scales_empty[turn.slot]));
    }
    turn.slots.next();
    if (ends && ++turn.slot == kGroups) {
      turn.slot = 0;
      turn.phase ^= 1;
    }
  }
  __device__ __forceinline__ void slab(int k) {
    begin(k);
#pragma unroll
    for (int c = 0; c < chunks; ++c) {
      tmem_ld_wait(r[c & 1]);
      const float4 x = now.x;
      const float w0 = now.w0, w1 = now.w1;
      if (c + 1 < chunks) {
        load(c + 1);
        now.x = *reinterpret_cast<const float4*>(now.as + 16 * (c + 1));
      } else {
        end(k);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t (&v)[8] = r[c & 1][h];
        const float2 w = h == 0 ? make_float2(w0, w0) : make_float2(w1, w1);
        float2 x0 = make_float2(x.x, x.y), x1 = make_float2(x.z, x.w);
        if (kind == kProdFwdSwiglu) {
          x0 = __fmul2_rn(x0, w);
          x1 = __fmul2_rn(x1, w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2& sum = a.v[c / 2][h][4 * (c & 1) + j];
          sum = __ffma2_rn(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), j < 2 ? x0 : x1, sum);
        }
      }
    }
  }
};

template <int kind, int chunks>
__device__ __forceinline__ void add_slabs(Sums& a, Shared& s, Turn& turn, uint32_t tmem, int half, int w, int lane, int slabs) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[c][h][j] = make_float2(0.0f, 0.0f);
  Turn at = turn;
  const int column = half * 16 * chunks;
  Adder<kind, chunks> add{a, s, at, tmem + column + (static_cast<uint32_t>(w * 32) << 16),
                          tc::in_block(tc::smem_addr(&s.acc_empty[0]), 0), lane, slabs, column, {}, {}};
#pragma unroll 1
  for (int k = 0; k < slabs; ++k) add.slab(k);
  turn = at;
}

template <typename T, int kind>
struct Epilogue {
  const F8Params& p;
  Shared& s;
  uint32_t* stage;  // of this half
  int rank, half, w, lane;

  // First row of the tile not to be stored, counted from the half's first.
  __device__ __forceinline__ int rows_left(const Tile& t, int c0) const { return t.cnt - t.r0 - c0; }

  // 16-bit words of two rows: staged[pair][feature], `features` of them, go to
  // rows c0 + 2 pair + {0, 1} of the tile.
  template <int features>
  __device__ __forceinline__ void store_pairs(const Tile& t, T* out, long long cols, int f, int width, int c0) const {
    constexpr int stride = features == kHalfM ? kPairStride : kGatedStride, per = 32 / (features / 4);
    const int l = lane & (features / 4 - 1), sub = lane / (features / 4);
    const int stop = f + 4 * l < width ? rows_left(t, c0) : 0;
    T* o = out + (static_cast<long long>(t.off) + t.r0 + c0) * cols + f + 4 * l;
#pragma unroll
    for (int i = 0; i < 4; i += per) {
      const int pair = 4 * w + i + sub;
      const uint4 q = *reinterpret_cast<const uint4*>(stage + pair * stride + 4 * l);
      if (2 * pair < stop)
        __stcs(reinterpret_cast<uint2*>(o + 2 * pair * cols), make_uint2(__byte_perm(q.x, q.y, 0x5410), __byte_perm(q.z, q.w, 0x5410)));
      if (2 * pair + 1 < stop)
        __stcs(reinterpret_cast<uint2*>(o + (2 * pair + 1) * cols), make_uint2(__byte_perm(q.x, q.y, 0x7632), __byte_perm(q.z, q.w, 0x7632)));
    }
  }

  __device__ __forceinline__ void plain(const Tile& t, const Sums& a, int nh) const {
    const int width = kind == kProdFwd ? p.N : p.K, f = t.f0 + rank * kHalfM;
    uint32_t* put = stage + (lane & 3) * kPairStride + w * 32 + (lane >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= nh) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 v = a.v[i][h][j];
          put[j / 2 * 4 * kPairStride + h * 16 + (j & 1) * 8] = pack2<T>(v.x, v.y);
        }
      half_sync(half);
      Tile part = t;
      part.cnt = min(t.cnt, t.r0 + (half + 1) * nh);  // past the half's columns lies the other half's
      store_pairs<kHalfM>(part, static_cast<T*>(p.out), width, f, width, half * nh + 32 * i);
      half_sync(half);
    }
  }

  // Sixteen rows at a time go through shared memory, unrounded; the gate and up
  // values of the next 32 are loaded meanwhile, the first ones before the slabs
  // are added (by `add`).
  template <typename Add>
  __device__ __forceinline__ void through_activation(const Tile& t, Sums& a, int nh, Add add) const {
    const int f = t.f0 + rank * kHalfM + 4 * lane;
    const long long cols = 2LL * p.K;
    float2* put = reinterpret_cast<float2*>(stage) + (lane & 3) * kPairStride32 + w * 32 + (lane >> 2);
    const int stop = f < p.K ? min(t.cnt - t.r0, (half + 1) * nh) : 0;
    const long long at0 = (static_cast<long long>(t.off) + t.r0 + half * nh + 4 * w) * cols + f;
    const T* pre = static_cast<const T*>(p.pre_in) + at0;
    T* out = static_cast<T*>(p.out) + at0;
    uint2 g[3][4], u[3][4];
    auto load = [&](int s, uint2 (&gs)[4], uint2 (&us)[4]) {
      const int c0 = half * nh + 16 * s + 4 * w;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (c0 + r < stop) {
          gs[r] = __ldg(reinterpret_cast<const uint2*>(pre + (16 * s + r) * cols));
          us[r] = __ldg(reinterpret_cast<const uint2*>(pre + (16 * s + r) * cols + p.K));
        }
    };
    load(0, g[0], u[0]);
    if (16 < nh) load(1, g[1], u[1]);
    add();
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (16 * s >= nh) break;
      const int c0 = half * nh + 16 * s + 4 * w;
      if (16 * (s + 2) < nh) load(s + 2, g[(s + 2) % 3], u[(s + 2) % 3]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) put[j / 2 * 4 * kPairStride32 + h * 16 + (j & 1) * 8] = a.v[s / 2][h][4 * (s & 1) + j];
      half_sync(half);
      float x[4][4];
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float2*>(stage) + (2 * w + r / 2) * kPairStride32 + 4 * lane);
        const float4 lo = q[0], hi = q[1];
        x[r][0] = lo.x; x[r + 1][0] = lo.y; x[r][1] = lo.z; x[r + 1][1] = lo.w;
        x[r][2] = hi.x; x[r + 1][2] = hi.y; x[r][3] = hi.z; x[r + 1][3] = hi.w;
      }
      half_sync(half);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (c0 + r < stop) {
          const float4 gv = unpack4<T>(g[s % 3][r]), uv = unpack4<T>(u[s % 3][r]);
          const float gs[4] = {gv.x, gv.y, gv.z, gv.w}, us[4] = {uv.x, uv.y, uv.z, uv.w};
          float dg[4], du[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float sg = fast_sigmoid(gs[k]);
            dg[k] = x[r][k] * us[k] * sg * (1.0f + gs[k] * (1.0f - sg));
            du[k] = x[r][k] * gs[k] * sg;
          }
          T* o = out + (16 * s + r) * cols;
          store4(o, make_float4(dg[0], dg[1], dg[2], dg[3]));
          store4(o + p.K, make_float4(du[0], du[1], du[2], du[3]));
        }
    }
  }

  // `turn`: which of the exchange's buffers this tile uses; `parity`: the phase of its barriers.
  __device__ __forceinline__ void gated(const Tile& t, Sums& a, int nh, int turn, uint32_t parity) const {
    const int F = p.N / 2, f = t.f0 + rank * (kHalfM / 2);
    Tile part = t;
    part.cnt = min(t.cnt, t.r0 + (half + 1) * nh);
    if (p.pre != nullptr) {
      uint32_t* put = stage + (lane & 3) * kGatedStride + w * 16 + (lane >> 2);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (32 * i >= nh) break;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 v = a.v[i][h][j];
            put[j / 2 * 4 * kGatedStride + (j & 1) * 8] = pack2<T>(v.x, v.y);
          }
          half_sync(half);
          store_pairs<kHalfM / 2>(part, static_cast<T*>(p.pre) + h * F, p.N, f, F, half * nh + 32 * i);
          half_sync(half);
        }
    }
    // The activation takes the place of the gate's sums.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= nh) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 g = a.v[i][0][j], u = a.v[i][1][j];
        a.v[i][0][j] = make_float2(g.x * fast_sigmoid(g.x) * u.x, g.y * fast_sigmoid(g.y) * u.y);
      }
    }
    if (p.out != nullptr) {
      uint32_t* put = stage + (lane & 3) * kGatedStride + w * 16 + (lane >> 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (32 * i >= nh) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 v = a.v[i][0][j];
          put[j / 2 * 4 * kGatedStride + (j & 1) * 8] = pack2<T>(v.x, v.y);
        }
        half_sync(half);
        store_pairs<kHalfM / 2>(part, static_cast<T*>(p.out), F, f, F, half * nh + 32 * i);
        half_sync(half);
      }
    }
    if (p.q == nullptr) return;
    // Largest magnitudes: over this warp's 16 features, the half's four warps,
    // then the other block's 64 features.
    float* most = reinterpret_cast<float*>(stage);  // [4 warps][128 columns], then [128]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= nh) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = a.v[i][0][2 * j], y = a.v[i][0][2 * j + 1];
        float m0 = max_nan(fabsf(x.x), fabsf(y.x)), m1 = max_nan(fabsf(x.y), fabsf(y.y));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          m0 = max_nan(m0, __shfl_xor_sync(0xffffffffu, m0, d));
          m1 = max_nan(m1, __shfl_xor_sync(0xffffffffu, m1, d));
        }
        if (lane < 4) *reinterpret_cast<float2*>(most + w * kHalfN + 32 * i + 8 * j + 2 * lane) = make_float2(m0, m1);
      }
    }
    half_sync(half);
    const int c = w * 32 + lane;  // a column of the half for each thread
    float m = 0.0f;
    if (c < nh) {
      m = max_nan(max_nan(most[c], most[kHalfN + c]), max_nan(most[2 * kHalfN + c], most[3 * kHalfN + c]));
      store_peer(tc::in_block(tc::smem_addr(&s.peer_max[turn][half * nh + c]), rank ^ 1), m);
    }
    half_sync(half);
    if (c == 0) tc::mbar_publish_cluster(tc::in_block(tc::smem_addr(&s.peer_full[turn][half]), rank ^ 1));
    tc::mbar_wait<true>(tc::smem_addr(&s.peer_full[turn][half]), parity, &s.gave_up);
    if (c < nh) {
      const BlockScale b = block_scale(max_nan(m, s.peer_max[turn][half * nh + c]));
      most[c] = b.inv;
      if (rank == 0 && c < part.cnt - t.r0 - half * nh) {
        float* qs = p.qs + (static_cast<long long>(t.off) + t.r0 + half * nh + c) * scale_columns(F) + t.f0 / kF8Block;
        qs[0] = b.scale;
        if (t.f0 + kF8Block >= F)
          for (int k = 1; t.f0 / kF8Block + k < scale_columns(F); ++k) qs[k] = 0.0f;
      }
    }
    half_sync(half);
    float2 inv[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= nh) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) inv[i][j] = *reinterpret_cast<const float2*>(most + 32 * i + 8 * j + 2 * (lane & 3));
    }
    half_sync(half);  // read: `most` gives way to the values
    // Two rows' bytes of a feature are a half word: staged[pair][64 features], 144 bytes apart.
    unsigned short* put = reinterpret_cast<unsigned short*>(stage) + (lane & 3) * 72 + w * 16 + (lane >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= nh) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 v = a.v[i][0][j];
        put[j / 2 * 4 * 72 + (j & 1) * 8] = static_cast<unsigned short>(e4m3x2(v.x * inv[i][j / 2].x, v.y * inv[i][j / 2].y));
      }
      half_sync(half);
      {
        const int pair = 4 * w + (lane >> 3), l = lane & 7, c0 = half * nh + 32 * i;
        const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(stage) + pair * 144 + 16 * l);
        uint8_t* o = p.q + (static_cast<long long>(t.off) + t.r0 + c0 + 2 * pair) * F + f + 8 * l;
        const int stop = part.cnt - t.r0 - c0;
        if (2 * pair < stop) __stcs(reinterpret_cast<uint2*>(o), make_uint2(__byte_perm(q.x, q.y, 0x6420), __byte_perm(q.z, q.w, 0x6420)));
        if (2 * pair + 1 < stop) __stcs(reinterpret_cast<uint2*>(o + F), make_uint2(__byte_perm(q.x, q.y, 0x7531), __byte_perm(q.z, q.w, 0x7531)));
      }
      half_sync(half);
    }
  }

  // Padding rows [cnt, rows) of the expert, the tile's features: zeros.
  __device__ __forceinline__ void zero_rows(const Tile& t) const {
    const int from = t.cnt + half * 4 + w;
    if constexpr (kind == kProdFwdSwiglu) {
      const int F = p.N / 2, f = t.f0 + rank * (kHalfM / 2) + 4 * (lane & 15);
      for (int r = from; r < t.rows; r += kEpilogueWarps) {
        const long long row = static_cast<long long>(t.off) + r;
        if (lane < 16) {
          if (p.out != nullptr) *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * F + f) = make_uint2(0, 0);
          if (p.q != nullptr) *reinterpret_cast<uint32_t*>(p.q + row * F + f) = 0;
        }
        if (p.pre != nullptr) *reinterpret_cast<uint2*>(static_cast<T*>(p.pre) + row * p.N + (lane >> 4) * F + f) = make_uint2(0, 0);
        if (p.q != nullptr && rank == 0 && t.f0 == 0)
          for (int b = lane; b < scale_columns(F); b += 32) p.qs[row * scale_columns(F) + b] = 0.0f;
      }
    } else {
      const int width = kind == kProdFwd ? p.N : p.K, f = t.f0 + rank * kHalfM + 4 * lane;
      if (f >= width) return;
      const long long cols = kind == kProdDgradSwiglu ? 2LL * width : width;
      for (int r = from; r < t.rows; r += kEpilogueWarps) {
        T* o = static_cast<T*>(p.out) + (static_cast<long long>(t.off) + r) * cols + f;
        *reinterpret_cast<uint2*>(o) = make_uint2(0, 0);
        if (kind == kProdDgradSwiglu) *reinterpret_cast<uint2*>(o + width) = make_uint2(0, 0);
      }
    }
  }
};

template <typename T, int kind>
__global__ void __launch_bounds__(kThreads, 1)
    ep_product_f8_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ CUtensorMap map_b64, const __grid_constant__ CUtensorMap map_b32,
                         const __grid_constant__ CUtensorMap map_b16, const __grid_constant__ CUtensorMap map_pre,
                         const F8Params p) {
  constexpr bool fwd = kind == kProdFwd || kind == kProdFwdSwiglu;
  extern __shared__ unsigned char raw[];
  unsigned char* ring = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  uint32_t* staging = reinterpret_cast<uint32_t*>(ring + kRingBytes);
  Shared& s = *reinterpret_cast<Shared*>(staging + 2 * kStageWords);
  // Through a shuffle the compiler knows that a warp shares the value: tensor
  // memory is addressed by uniform registers, and each conversion to one costs.
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(tc::cluster_rank());
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map_a);
    tc::tma_prefetch_desc(&map_b);
    tc::tma_prefetch_desc(&map_b16);
    for (int i = 0; i < kMaxStages; ++i) {
      tc::mbar_init(tc::smem_addr(&s.full[i]), 2);  // the first block's two loaders account for both blocks' copies
      tc::mbar_init(tc::smem_addr(&s.empty[i]), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      tc::mbar_init(tc::smem_addr(&s.acc_full[i]), 1);
      tc::mbar_init(tc::smem_addr(&s.acc_empty[i]), 2 * kEpilogueWarps);
    }
    for (int i = 0; i < kExchanges; ++i)
      for (int j = 0; j < 2; ++j) tc::mbar_init(tc::smem_addr(&s.peer_full[i][j]), 1);
    for (int i = 0; i < kGroups; ++i) {
      tc::mbar_init(tc::smem_addr(&s.scales_full[i]), 32);
      tc::mbar_init(tc::smem_addr(&s.scales_empty[i]), kEpilogueWarps);
    }
    tc::mbar_init(tc::smem_addr(&s.drained), 1);
    tc::mbar_init_fence();
    s.gave_up = s.most = 0;
  }
  if (warp == 2) tc::tmem_alloc(tc::smem_addr(&s.tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
  pdl_wait();
  if (threadIdx.x == 0) s.ok = blocks_ok(p.hdr, p.R);
  __syncthreads();
  const bool ok = s.ok;
  if (ok) scan_row_blocks(p, s.cum, s.part, &s.most);
  const int stage_bytes = kABytes + box_rows((min(s.most, kTileN) + 31) / 32 * 16) * kSlab;
  const int stages = min(kMaxStages, kRingBytes / stage_bytes);
  const int red = fwd ? p.K : p.N, slabs = (red + kSlab - 1) / kSlab;
  volatile int* gave_up = &s.gave_up;
  const long long first = blockIdx.x / 2, step = gridDim.x / 2;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (ok) {
      Walk<kind> walk(p, s.cum);
      Tile t;
      if (warp == 0 || warp == 2) {
        if (lane == 0) {
          const bool load_a = warp == 0;
          int stage = 0;
          uint32_t phase = 0;
          for (long long i = first; i < walk.total && !*gave_up; i += step) {
            walk.at(i, &t);
            const int half = t.n / 2;  // this block's rows
            const int bytes = load_a ? kABytes : box_rows(half) * kSlab;
            for (int k = 0; k < slabs; ++k) {
              if (!tc::mbar_wait(tc::smem_addr(&s.empty[stage]), phase ^ 1, gave_up)) break;
              const uint32_t a = tc::smem_addr(ring + static_cast<size_t>(stage) * stage_bytes), b = a + kABytes;
              const uint32_t bar = rank == 0 ? tc::smem_addr(&s.full[stage]) : tc::in_block(tc::smem_addr(&s.full[stage]), 0);
              if (rank == 0) tc::mbar_expect(bar, 2 * bytes);  // the other block's copies too
              const int x = k * kSlab;
              if constexpr (kind == kProdDgradSwiglu) {
                // The gate and up values that the tile's end reads go to L2 while
                // its last slabs are added (what the other blocks then read and
                // write at the same time): 297 us without, 295 twelve slabs from
                // the end, 273 here.
                const int f = t.f0 + rank * kHalfM;
                if (!load_a && k == max(0, slabs - 3) && f < p.K)
                  for (int r = 0; r < t.n; r += 128) {
                    prefetch_2d(&map_pre, 2 * f, t.off + t.r0 + r);
                    prefetch_2d(&map_pre, 2 * (f + p.K), t.off + t.r0 + r);
                  }
              }
              if (load_a) {
                if constexpr (kind == kProdFwd) {
                  tc::tma_pair_3d(a, &map_a, bar, x, t.f0 + rank * kHalfM, t.e);
                } else if constexpr (kind == kProdFwdSwiglu) {
                  // four times 16 gate rows, then the up rows of the same features
                  tc::tma_pair_5d(a, &map_a, bar, x, 0, 0, (t.f0 + rank * (kHalfM / 2)) / 16, t.e);
                } else {
                  tc::tma_pair_3d(a, &map_a, bar, t.f0 + rank * kHalfM, x, t.e);
                }
              } else {
                tc::tma_pair_2d(b, half > 64 ? &map_b : half > 32 ? &map_b64 : half > 16 ? &map_b32 : &map_b16, bar, x,
                                t.off + t.r0 + rank * half);
              }
              if (++stage == stages) {
                stage = 0;
                phase ^= 1;
              }
            }
          }
          if (load_a) pdl_trigger();
          // Every stage is read out before the block ends.
          for (int j = 0; j < stages && !*gave_up; ++j) {
            if (!tc::mbar_wait(tc::smem_addr(&s.empty[stage]), phase ^ 1, gave_up)) break;
            if (++stage == stages) {
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
      } else if (warp == 1) {
        if (rank == 0) {
          int stage = 0;
          uint32_t phase = 0;
          Slots slots;
          bool lost = false;
          const uint32_t ring0 = tc::smem_addr(ring), full0 = tc::smem_addr(&s.full[0]), empty0 = tc::smem_addr(&s.empty[0]);
          const uint32_t acc_full0 = tc::smem_addr(&s.acc_full[0]), acc_empty0 = tc::smem_addr(&s.acc_empty[0]);
          for (long long i = first; i < walk.total && !lost; i += step) {
            walk.at(i, &t);
            t.n = __shfl_sync(0xffffffffu, t.n, 0);
            const uint32_t desc = mma_desc_f8(!fwd, kTileM, t.n);
            if (Slots::of(t.n) != slots.width) {
              // The slots were others' parts: all of those are read out first.
              for (int j = 0; slots.width > 0 && j < kSlots; j += slots.width)
                lost = lost || !warp_wait(acc_empty0 + 8 * j, (slots.phases >> j & 1) ^ 1, gave_up);
              slots.width = Slots::of(t.n);
              slots.at = 0;
            }
            for (int k = 0; k < slabs && !lost; ++k) {
              lost = !warp_wait(acc_empty0 + 8 * slots.at, slots.phase() ^ 1, gave_up) || !warp_wait(full0 + 8 * stage, phase, gave_up);
              if (lost) break;
              tc::fence_after();
              // What lies past the reduction's end came as zeros.
              const uint32_t a = ring0 + stage * stage_bytes;
              mma_slab<fwd ? tc::kDescStepK : kDescStepMn8>(tmem + slots.at * kSlotColumns,
                                                           fwd ? tc::desc_k_major(a) : tc::desc_mn_major(a, kABytes),
                                                           tc::desc_k_major(a + kABytes), desc, empty0 + 8 * stage, acc_full0 + 8 * slots.at);
              if (++stage == stages) {
                stage = 0;
                phase ^= 1;
              }
              slots.next();
            }
          }
          if (lost && elect()) {
            // What was issued ends before tensor memory is freed.
            tc::mma_commit(tc::smem_addr(&s.drained));
            const unsigned long long start = tc::now_ns();
            while (!tc::mbar_try(tc::smem_addr(&s.drained), 0) && tc::now_ns() - start < tc::kWaitNs) {
            }
          }
        }
      } else {
        // Scales of four slabs: lane l brings rows l, l + 32, ...
        int slot = 0;
        uint32_t phase = 0;
        const int cols = scale_columns(red), kb = f8_blocks(p.K), nb = f8_blocks(p.N);
        for (long long i = first; i < walk.total && !*gave_up; i += step) {
          walk.at(i, &t);
          const int row0 = t.off + t.r0;
          const int fb = min((t.f0 + (kind == kProdFwdSwiglu ? rank * (kHalfM / 2) : rank * kHalfM)) / kF8Block, (fwd ? nb : kb) - 1);
          const float* ws = p.ws + static_cast<long long>(t.e) * nb * kb;
          for (int k = 0; k < slabs; k += kGroup) {
            float4 v[kTileN / 32];
#pragma unroll
            for (int j = 0; j < kTileN / 32; ++j) {
              const int r = j * 32 + lane;
              v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (r < t.n && row0 + r < p.R) v[j] = __ldg(reinterpret_cast<const float4*>(p.as + static_cast<long long>(row0 + r) * cols + k));
            }
            float w = 0.0f;
            const int b = k + (lane & 3), up = lane >> 2;  // lanes 4 to 7: the up rows' scales
            if (up < (kind == kProdFwdSwiglu ? 2 : 1) && b < slabs)
              w = __ldg(ws + (fwd ? static_cast<long long>(fb + up * (nb / 2)) * kb + b : static_cast<long long>(b) * kb + fb));
            if (!warp_wait(tc::smem_addr(&s.scales_empty[slot]), phase ^ 1, gave_up)) break;
            // Of 16 rows, those of one quarter of a warp's lanes (2 l, 2 l + 1,
            // and 8 further on) lie side by side.
            const int to = (lane & 16) + (lane & 6) * 2 + (lane & 8) / 4 + (lane & 1);
            float w4[kGroup];
#pragma unroll
            for (int q = 0; q < kGroup; ++q) w4[q] = kind == kProdFwdSwiglu ? 1.0f : __shfl_sync(0xffffffffu, w, q);
#pragma unroll
            for (int j = 0; j < kTileN / 32; ++j) {
              s.as[slot][0][j * 32 + to] = v[j].x * w4[0];
              s.as[slot][1][j * 32 + to] = v[j].y * w4[1];
              s.as[slot][2][j * 32 + to] = v[j].z * w4[2];
              s.as[slot][3][j * 32 + to] = v[j].w * w4[3];
            }
            if (kind == kProdFwdSwiglu && lane < 8) s.ws[slot][up][lane & 3] = w;
            tc::mbar_arrive(tc::smem_addr(&s.scales_full[slot]));
            if (++slot == kGroups) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    if (ok) {
      Walk<kind> walk(p, s.cum);
      Tile t;
      const int half = (warp - 4) >> 2, w = warp & 3;  // the accumulator lanes a warp can reach go by its number
      const Epilogue<T, kind> out{p, s, staging + half * kStageWords, rank, half, w, lane};
      int turn = 0;
      uint32_t peer_phase = 0;
      Turn at;
      for (long long i = first; i < walk.total; i += step) {
        walk.at(i, &t);
        t.n = __shfl_sync(0xffffffffu, t.n, 0);
        const int nh = t.n / 2;
        if (Slots::of(t.n) != at.slots.width) {
          at.slots.width = Slots::of(t.n);
          at.slots.at = 0;
        }
        Sums a;
        auto add = [&]() {
          switch (nh / 16) {
            case 1: add_slabs<kind, 1>(a, s, at, tmem, half, w, lane, slabs); break;
            case 2: add_slabs<kind, 2>(a, s, at, tmem, half, w, lane, slabs); break;
            case 3: add_slabs<kind, 3>(a, s, at, tmem, half, w, lane, slabs); break;
            case 4: add_slabs<kind, 4>(a, s, at, tmem, half, w, lane, slabs); break;
            case 5: add_slabs<kind, 5>(a, s, at, tmem, half, w, lane, slabs); break;
            case 6: add_slabs<kind, 6>(a, s, at, tmem, half, w, lane, slabs); break;
            case 7: add_slabs<kind, 7>(a, s, at, tmem, half, w, lane, slabs); break;
            default: add_slabs<kind, 8>(a, s, at, tmem, half, w, lane, slabs); break;
          }
        };
        if constexpr (kind != kProdDgradSwiglu) add();
        if constexpr (kind == kProdFwdSwiglu) {
          out.gated(t, a, nh, turn, peer_phase);
          if (++turn == kExchanges) {
            turn = 0;
            peer_phase ^= 1;
          }
        } else if constexpr (kind == kProdDgradSwiglu) {
          out.through_activation(t, a, nh, add);
        } else {
          out.plain(t, a, nh);
        }
        if (t.last) out.zero_rows(t);
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

// A map of [dim 4]..[dim 1][dim 0] bytes.
bool make_map(CUtensorMap* m, const void* base, int dims, const long long (&size)[5], const long long (&stride)[4],
              const int (&box)[5], bool swizzle = true) {
  const tc::EncodeFn f = tc::tensor_map_encoder();
  if (f == nullptr) return false;
  cuuint64_t sz[5], st[4];
  cuuint32_t bx[5];
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < dims; ++i) {
    sz[i] = static_cast<cuuint64_t>(size[i]);
    bx[i] = static_cast<cuuint32_t>(box[i]);
    if (i + 1 < dims) st[i] = static_cast<cuuint64_t>(stride[i]);
  }
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(dims), const_cast<void*>(base), sz, st, bx, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of blocks that fit on the current device at once (0: the query
// failed); the kernel's shared memory is raised on the way.  Once per device.
template <typename T, int kind>
int resident_pairs(int num_sms) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int pairs = known[dev].load(std::memory_order_acquire);
  if (pairs == 0) {
    const auto kern = ep_product_f8_kernel<T, kind>;
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

template <typename T, int kind>
cudaError_t launch_kind(const F8Params& p, int num_sms, cudaStream_t s) {
  CUtensorMap a, b, b64, b32, b16, pre = {};
  constexpr bool fwd = kind == kProdFwd || kind == kProdFwdSwiglu;
  const long long K = p.K, N = p.N, red = fwd ? K : N, F = N / 2;
  bool ok = kind == kProdFwdSwiglu
                ? make_map(&a, p.w, 5, {K, 16, 2, F / 16, p.E}, {K, F * K, 16 * K, 2 * F * K}, {kSlab, 16, 2, 4, 1})
                : make_map(&a, p.w, 3, {K, N, p.E, 1, 1}, {K, N * K, 0, 0}, {kSlab, 128, 1, 1, 1});
  CUtensorMap* maps[4] = {&b, &b64, &b32, &b16};
  for (int i = 0; i < 4; ++i) ok = ok && make_map(maps[i], p.a, 2, {red, p.R, 1, 1, 1}, {red, 0, 0, 0}, {kSlab, 128 >> i, 1, 1, 1});
  if (kind == kProdDgradSwiglu)  // 128 features of 128 rows
    ok = ok && make_map(&pre, p.pre_in, 2, {4 * K, p.R, 1, 1, 1}, {4 * K, 0, 0, 0}, {256, 128, 1, 1, 1}, false);
  if (!ok) return cudaErrorInvalidValue;
  const int pairs = resident_pairs<T, kind>(num_sms);
  if (pairs == 0) return cudaErrorLaunchOutOfResources;
  return launch_pdl(ep_product_f8_kernel<T, kind>, dim3(2 * pairs), dim3(kThreads), kSmemBytes, s, 2, a, b, b64, b32, b16, pre, p);
}

template <typename T>
cudaError_t launch_typed(const F8Params& p, int num_sms, cudaStream_t s) {
  switch (p.kind) {
    case kProdFwd: return launch_kind<T, kProdFwd>(p, num_sms, s);
    case kProdFwdSwiglu: return launch_kind<T, kProdFwdSwiglu>(p, num_sms, s);
    case kProdDgrad: return launch_kind<T, kProdDgrad>(p, num_sms, s);
    default: return launch_kind<T, kProdDgradSwiglu>(p, num_sms, s);
  }
}

}  // namespace

cudaError_t launch_product_f8(const F8Params& p, int num_sms, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP16) return launch_typed<__half>(p, num_sms, s);
  return launch_typed<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace ep
