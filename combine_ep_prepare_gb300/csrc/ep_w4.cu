// ep_w4.cu -- products of a few rows per expert with 4-bit weights.
//
// w[e][n][k] = scales[e][n][k / group] * (q - 8), q the unsigned nibble k of
// row n (low nibble of a byte: even k).  out[r][n] = sum_k x[r][k] w[e][n][k]
// for the rows of expert e, or silu(gate) * up of the two halves of n.
//
// The logic unit has most to do, 68% of its rate on a decode batch's down
// products (64 experts, 8 rows each, 2048 -> 7168): 54 M warp instructions,
// near 60 for a step of 32 weight rows x 32 elements, of which the unpacking is
// 28 and the rows' order, addresses and scales are the rest.  No unit is busier.
// Those products take 141 us; without the unpacking 90, without the copies
// 131, and memory alone would take 73.
//
// Two persistent blocks per SM walk units of 256 down to 64 weight rows of one
// expert: one warp keeps a ring of two 32 KB stages filled by TMA (and the
// receive rows' share with them), running ahead across units; of eight others
// each owns 32 weight rows and a share of the reduction.  Where there are few
// units, 2 or 4 warps share 32 rows and split the reduction, joined through
// shared memory in a fixed order.  One block of eight consumers per SM took
// 148 us for those down products: two warps a scheduler do not hide each
// other's latencies.  A stage is 256 rows of 128 bytes (256 weights): the
// copies cost a block about two clocks a row, so 64-byte rows would not keep
// up with memory, and copies of 16 or 32 rows for each warp cost 90 clocks
// each to issue (20 to 32 of them a stage: 188 us).  cp.async by the consumers
// themselves costs 40% more instructions (169 us).
//
// The receive rows are the narrow side of mma.m16n8k16 (weights 16 x 16,
// receive rows 16 x 8): up to 16 rows share one pass over the weights.  A
// nibble becomes an integer plus a constant by being placed in the mantissa
// of a 16-bit number, one packed operation gives q - 8 exactly, and the
// integers' sum over a group is exact up to the float32 accumulation of q x;
// the scale multiplies that sum in float32, so no weight is ever rounded.
// The weights are unpacked again for every 16 rows: from 33 rows per expert on
// the 16-bit product is faster (16 experts, 2048 -> 7168: 76 us against 79 at
// 32 rows each, 123 against 81 at 48, 294 against 84 at 128).
#include "ep_experts.cuh"
#include "ep_tc.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;                     // consumers; one more warp loads
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kBoxRows = 32, kChunk = 256;    // a warp's weight rows and reduction elements per stage
constexpr int kRowBytes = kChunk / 2;
constexpr int kBoxBytes = kBoxRows * kRowBytes;
constexpr int kWBytes = kWarps * kBoxBytes;
constexpr int kSlabBytes = 8 * kChunk * 2;    // eight receive rows' share of a stage
constexpr int kMaxSlabs = 4;                  // shares times blocks of eight rows
constexpr int kStageBytes = kWBytes + kMaxSlabs * kSlabBytes;
constexpr int kStages = 2;
constexpr int kSteps = kChunk / 32;           // steps of 32 reduction elements
constexpr int kUnitRows = kWarps * kBoxRows;
constexpr int kMaxSplit = 4;

// The eight nibbles of a word, as the pairs (0,4) (1,5) (2,6) (3,7) of q - 8:
// nibbles i and i + 4 lie 16 bits apart, so one shift and one mask place both.
// The logic unit, which takes an instruction every other clock, has most of
// the kernel's work here.  (Shifts by the multipliers' upper halves instead
// took 190 us for 173 on a decode batch's down products.)
template <typename T>
struct Nib;
template <>
struct Nib<__nv_bfloat16> {
  // 128 + q, less 136
  static __device__ __forceinline__ void unpack(unsigned w, unsigned (&out)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
      asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(out[i]) : "r"(v), "r"(0xc308c308u));
    }
  }
  // c = a b
  static __device__ __forceinline__ void mma0(float* c, const unsigned* a, unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  }
  static __device__ __forceinline__ void mma(float* c, const unsigned* a, unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Nib<__half> {
  // Even nibbles as 1024 + q, less 1032; odd ones where they are, 1024 + 16 q,
  // over 16 less 72: exact, and without a shift.
  static __device__ __forceinline__ void unpack(unsigned w, unsigned (&out)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const unsigned s = w >> (4 * i);
      const unsigned even = (s & 0x000f000fu) | 0x64006400u, odd = (s & 0x00f000f0u) | 0x64006400u;
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(out[i]) : "r"(even), "r"(0xe408e408u));
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(out[i + 1]) : "r"(odd), "r"(0x2c002c00u), "r"(0xd480d480u));
    }
  }
  // c = a b
  static __device__ __forceinline__ void mma0(float* c, const unsigned* a, unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  }
  static __device__ __forceinline__ void mma(float* c, const unsigned* a, unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// A unit: kUnitRows / KW weight rows of an expert times a block of 8 nt rows.
struct Unit {
  int e, n0, r0, cnt, off, nt, kw;
  bool last;  // the expert's last row block: zeroes the padding rows
};

struct Blocks {
  int nt, kw, nblk, tblk;
  __device__ __forceinline__ Blocks(const W4Params& p, int cnt, int KW) {
    nt = cnt <= 8 ? 1 : 2;
    kw = KW < kMaxSlabs / nt ? KW : kMaxSlabs / nt;
    const int rows = kUnitRows / kw;
    nblk = (p.N + rows - 1) / rows;  // gated: N / 2 features over rows / 2
    tblk = (cnt + 8 * nt - 1) / (8 * nt);
  }
};

struct Shared {
  uint64_t full[kStages], empty[kStages];
  int gave_up, ok, stop;
  int part[32];
  int cum[EP_MAX_EXPERTS + 1];  // units of the experts before e
};
constexpr int kScaleBytes = kWarps * kBoxRows * 16;              // 256 / 32 scales of every box row
constexpr int kRedBytes = kWarps / kMaxSplit * (kMaxSplit - 1) * 32 * 8 * 4;  // sums of 8 rows of all but one share
constexpr size_t kSmemBytes =
    static_cast<size_t>(kStages) * kStageBytes + kScaleBytes + kRedBytes + 1024 + sizeof(Shared);

// cum[e] = units of the experts before e when the reduction is split KW ways.
__device__ __forceinline__ void scan_units(const W4Params& p, int KW, Shared& s) {
  int base = 0;
  for (int e0 = 0; e0 < p.E; e0 += kThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int cnt = e < p.E ? p.counts[e] : 0;
    const Blocks b(p, cnt, KW);
    const int v = block_scan<kThreads>(cnt > 0 ? b.nblk * b.tblk : 0, s.part);
    if (e < p.E) s.cum[e + 1] = base + v;
    if (threadIdx.x == kThreads - 1) s.part[0] = v;
    __syncthreads();
    base += s.part[0];
    __syncthreads();
  }
  if (threadIdx.x == 0) s.cum[0] = 0;
  __syncthreads();
}

// o->e: the expert to search from.
__device__ __forceinline__ void unit_at(const W4Params& p, const Shared& s, int KW, int u, Unit* o) {
  while (u >= s.cum[o->e + 1]) ++o->e;
  o->cnt = p.counts[o->e];
  o->off = p.offsets[o->e];
  const Blocks b(p, o->cnt, KW);
  const int in = u - s.cum[o->e], tb = in % b.tblk;
  o->nt = b.nt;
  o->kw = b.kw;
  o->n0 = in / b.tblk * (kUnitRows / b.kw);
  o->r0 = tb * 8 * b.nt;
  o->last = tb + 1 == b.tblk;
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

// Shared memory from its first 1024-byte boundary.
__device__ __forceinline__ unsigned char* block_smem() {
  extern __shared__ unsigned char raw[];
  return raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
}

// What a consumer warp keeps over the units.
template <typename T, int G, bool gated>
struct Consumer {
  const W4Params& p;
  Shared& s;
  int chunks, warp, lane;
  int stage;
  uint32_t phase;

  // One unit's sums.  False when a wait gave up.
  template <int NT>
  __device__ __forceinline__ bool sums(const Unit& u, float (&total)[2][NT][4]) {
    const int g = lane >> 2, t = lane & 3, KW = u.kw, sub = warp % KW, group = warp / KW;
    const int iters = (chunks + KW - 1) / KW;
    constexpr int kGroups = kChunk / G;
    int left = min(p.K - sub * iters * kChunk, iters * kChunk);  // elements of the warp's share
    // Scales: lane l brings a stage's scales of box row l, a stage ahead, and
    // the warp shares them through shared memory, eight words' space a row.
    const T* scale;
    int groups_left = p.K / G - sub * iters * kGroups;
    {
      int n;  // weight row of box row `lane`, clamped into the expert
      if (gated) {
        const int F = p.N / 2;
        n = min(u.n0 / 2 + group * 16 + (lane & 15), F - 1) + (lane >> 4) * F;
      } else {
        n = min(u.n0 + group * kBoxRows + lane, p.N - 1);
      }
      scale = static_cast<const T*>(p.scales) + (static_cast<long long>(u.e) * p.N + n) * (p.K / G) + sub * iters * kGroups;
    }
    const bool wide = p.K % kChunk == 0;  // rows of whole stages: a stage's scales lie on their own alignment
    uint32_t next[kGroups / 2];
    auto load_scales = [&]() {
#pragma unroll
      for (int i = 0; i < kGroups / 2; ++i) next[i] = 0;
      if (wide && groups_left > 0) {
        if constexpr (kGroups == 2) {
          next[0] = __ldg(reinterpret_cast<const uint32_t*>(scale));
        } else if constexpr (kGroups == 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(scale));
          next[0] = v.x;
          next[1] = v.y;
        } else {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(scale));
          next[0] = v.x;
          next[1] = v.y;
          next[2] = v.z;
          next[3] = v.w;
        }
      } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(scale);
#pragma unroll
        for (int q = 0; q < kGroups; ++q)
          if (q < groups_left) next[q / 2] |= static_cast<uint32_t>(__ldg(h + q)) << (16 * (q & 1));
      }
      scale += kGroups;
      groups_left -= kGroups;
    };
    unsigned char* smem = block_smem();
    unsigned char* scales = smem + kStages * kStageBytes + warp * (kBoxRows * 16);
    load_scales();
    float acc[2][NT][4], sc[2][2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[f][i][j] = 0.0f;
    }
    auto apply = [&]() {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) total[f][i][j] = fmaf(sc[f][j >> 1], acc[f][i][j], total[f][i][j]);
    };
    // Fragment f's rows g and g + 8 (gated: the gate row and the up row of one
    // feature) in the stage: this warp's rows of its share's box; the gate
    // rows of a box come before its up rows.
    const int sub_bytes = kWBytes / KW;
    const uint32_t word_at = sub * sub_bytes + group * (gated ? 16 : kBoxRows) * kRowBytes + g * kRowBytes + t * 4;
    const uint32_t h_bytes = gated ? sub_bytes / 2 : 8 * kRowBytes;
    constexpr int kFBytes = (gated ? 8 : 16) * kRowBytes;
    constexpr int kScaleF = (gated ? 8 : 16) * 16, kScaleH = (gated ? 16 : 8) * 16;  // box rows in the scales' order
    for (int it = 0; it < iters; ++it) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kGroups / 2; ++i) reinterpret_cast<uint32_t*>(scales + lane * 16)[i] = next[i];
      if (it + 1 < iters) load_scales();
      if (!__all_sync(0xffffffffu, tc::mbar_wait(tc::smem_addr(&s.full[stage]), phase, &s.gave_up))) return false;
      __syncwarp();  // the scales of all lanes are there: a vote orders no memory
      const unsigned char* words = smem + stage * kStageBytes + word_at;
      const unsigned char* slab = smem + stage * kStageBytes + kWBytes + sub * NT * kSlabBytes + g * (kChunk * 2);
#pragma unroll
      for (int kb = 0; kb < kSteps; ++kb) {
        // Rows' elements in the order of the nibble pairs: lane (g, t) has
        // eight from t * 8 of this run of 32 of row g of a slab.
        unsigned b[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              slab + i * kSlabBytes + kb * 64 + ((t ^ (kb >> 1)) << 4));
          b[i][0] = __byte_perm(v.x, v.z, 0x5410);
          b[i][1] = __byte_perm(v.x, v.z, 0x7632);
          b[i][2] = __byte_perm(v.y, v.w, 0x5410);
          b[i][3] = __byte_perm(v.y, v.w, 0x7632);
        }
        const unsigned char* w0 = words + ((kb ^ g) << 4);
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          unsigned a[2][4];
          Nib<T>::unpack(*reinterpret_cast<const unsigned*>(w0 + f * kFBytes), a[0]);
          Nib<T>::unpack(*reinterpret_cast<const unsigned*>(w0 + h_bytes + f * kFBytes), a[1]);
          const unsigned lo[4] = {a[0][0], a[1][0], a[0][1], a[1][1]}, hi[4] = {a[0][2], a[1][2], a[0][3], a[1][3]};
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (kb * 32 % G == 0) Nib<T>::mma0(acc[f][i], lo, b[i][0], b[i][1]);
            else Nib<T>::mma(acc[f][i], lo, b[i][0], b[i][1]);
            Nib<T>::mma(acc[f][i], hi, b[i][2], b[i][3]);
          }
        }
        if ((kb + 1) * 32 % G == 0) {
          const T* at_g = reinterpret_cast<const T*>(scales + g * 16) + kb * 32 / G;
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            sc[f][0] = to_f32(at_g[f * kScaleF / 2]);
            sc[f][1] = to_f32(at_g[(f * kScaleF + kScaleH) / 2]);
          }
          if (kb * 32 < left) apply();  // past the share's end: another share's rows, or none
        }
      }
      left -= kChunk;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_addr(&s.empty[stage]));
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    return true;
  }

  // Joins the reduction's shares (in ascending order, eight rows at a time)
  // and writes the unit's output.
  template <int NT>
  __device__ __forceinline__ void write(const Unit& u, float (&total)[2][NT][4]) {
    const int g = lane >> 2, t = lane & 3, KW = u.kw, sub = warp % KW, group = warp / KW;
    if (KW > 1) {
      float* red = reinterpret_cast<float*>(block_smem() + kStages * kStageBytes + kScaleBytes) + group * (KW - 1) * 256;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (sub > 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) red[(sub - 1) * 256 + j * 32 + lane] = total[j / 4][i][j % 4];
        }
        consumers_sync();
        if (sub == 0)
          for (int k = 0; k + 1 < KW; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) total[j / 4][i][j % 4] += red[k * 256 + j * 32 + lane];
          }
        consumers_sync();
      }
      if (sub > 0) return;
    }
    const int cols = gated ? p.N / 2 : p.N;
    T* out = static_cast<T*>(p.out) + static_cast<long long>(u.off) * cols;
    const int c0 = gated ? u.n0 / 2 + group * 16 : u.n0 + group * kBoxRows;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = u.r0 + i * 8 + 2 * t + j;
          if (r >= u.cnt) continue;
          if (gated) {
            const int c = c0 + f * 8 + g;
            if (c < cols) out[static_cast<long long>(r) * cols + c] = from_f32<T>(swiglu(total[f][i][j], total[f][i][2 + j]));
          } else {
            const int c = c0 + f * 16 + g;
            if (c < cols) out[static_cast<long long>(r) * cols + c] = from_f32<T>(total[f][i][j]);
            if (c + 8 < cols) out[static_cast<long long>(r) * cols + c + 8] = from_f32<T>(total[f][i][2 + j]);
          }
        }
    if (u.last) {
      const int c = c0 + lane;
      if (c < cols && lane < (gated ? 16 : kBoxRows))
        for (int r = u.cnt, rows = p.offsets[u.e + 1] - u.off; r < rows; ++r)
          out[static_cast<long long>(r) * cols + c] = from_f32<T>(0.0f);
    }
  }

  template <int NT>
  __device__ __forceinline__ bool unit(const Unit& u) {
    float total[2][NT][4];
    const bool fine = sums<NT>(u, total);
    if (fine || u.kw > 1) write<NT>(u, total);  // a split unit's barriers want every warp
    return fine;
  }
};

struct Maps {
  CUtensorMap box[3];  // weights in boxes of kUnitRows, / 2 or / 4 rows of kRowBytes (gated: half of each)
  CUtensorMap rows;    // receive rows, boxes of 8 rows x kChunk
};

template <typename T, int G, bool gated>
__global__ void __launch_bounds__(kThreads, 2) ep_w4_kernel(const __grid_constant__ Maps maps, const W4Params p) {
  unsigned char* smem = block_smem();
  Shared& s = *reinterpret_cast<Shared*>(smem + kStages * kStageBytes + kScaleBytes + kRedBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(tc::smem_addr(&s.full[i]), 1);
      tc::mbar_init(tc::smem_addr(&s.empty[i]), kWarps);
    }
    tc::mbar_init_fence();
    s.gave_up = 0;
    s.stop = 0;
  }
  pdl_wait();
  if (threadIdx.x == 0) s.ok = blocks_ok(p.hdr, p.R);
  __syncthreads();
  if (!s.ok) return;
  // The reduction is split until there is a unit for every block.
  const int chunks = (p.K + kChunk - 1) / kChunk;
  scan_units(p, 1, s);
  int KW = 1;
  while (KW < kMaxSplit && 2 * KW <= chunks && s.cum[p.E] * KW < static_cast<int>(gridDim.x)) KW *= 2;
  __syncthreads();
  if (KW > 1) scan_units(p, KW, s);
  const int total_units = s.cum[p.E];
  Unit u;
  u.e = 0;
  volatile int* gave_up = &s.gave_up;
  if (warp == kWarps) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int i = blockIdx.x; i < total_units && !*gave_up; i += gridDim.x) {
        unit_at(p, s, KW, i, &u);
        // A share's weight rows of a stage are one copy; gated two, gate rows first.
        const int boxes = (gated ? 2 : 1) * u.kw, rows = kUnitRows / boxes, iters = (chunks + u.kw - 1) / u.kw;
        const CUtensorMap* map = &maps.box[31 - __clz(u.kw)];
        for (int it = 0; it < iters; ++it) {
          if (!tc::mbar_wait(tc::smem_addr(&s.empty[stage]), phase ^ 1, gave_up)) break;
          const uint32_t full = tc::smem_addr(&s.full[stage]), dst = tc::smem_addr(smem + stage * kStageBytes);
          tc::mbar_expect(full, kWBytes + u.kw * u.nt * kSlabBytes);
          for (int b = 0; b < boxes; ++b) {
            const int share = gated ? b / 2 : b;
            const int row = gated ? (b & 1) * (p.N / 2) + u.n0 / 2 : u.n0;
            tc::tma_load_3d(dst + b * rows * kRowBytes, map, full, (share * iters + it) * kRowBytes, row, u.e);
          }
          for (int b = 0; b < u.kw * u.nt; ++b)
            tc::tma_load_3d(dst + kWBytes + b * kSlabBytes, &maps.rows, full, 0, (b / u.nt * iters + it) * kSteps,
                            u.off + u.r0 + b % u.nt * 8);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else {
    Consumer<T, G, gated> c{p, s, chunks, warp, lane, 0, 0};
    for (int i = blockIdx.x; i < total_units; i += gridDim.x) {
      unit_at(p, s, KW, i, &u);
      const bool fine = u.nt == 1 ? c.template unit<1>(u) : c.template unit<2>(u);
      if (KW > 1) {
        // All warps leave together, or the next unit's barriers would wait for one that left.
        if (threadIdx.x == 0) s.stop = *gave_up;
        consumers_sync();
        if (s.stop) break;
      } else if (!fine) {
        break;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && s.gave_up) {
    // Whoever gave up, the loading warp may have left before: the copies in
    // flight land before the block's shared memory goes; a copy takes
    // microseconds.
    const unsigned long long start = tc::now_ns();
    while (tc::now_ns() - start < tc::kWaitNs / 100) {
    }
    atomicOr(&p.hdr[kHdrStatus], static_cast<int>(EP_ST_TIMEOUT));
  }
}

template <typename T, int G, bool gated>
cudaError_t launch_one(const W4Params& p, const Maps& maps, int num_sms, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(ep_w4_kernel<T, G, gated>),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(ep_w4_kernel<T, G, gated>, dim3(2 * num_sms), dim3(kThreads), kSmemBytes, s, 0, maps, p);
}

template <typename T>
cudaError_t launch_typed(const W4Params& p, const Maps& maps, int num_sms, cudaStream_t s) {
  if (p.swiglu)
    return p.group == 32   ? launch_one<T, 32, true>(p, maps, num_sms, s)
           : p.group == 64 ? launch_one<T, 64, true>(p, maps, num_sms, s)
                           : launch_one<T, 128, true>(p, maps, num_sms, s);
  return p.group == 32   ? launch_one<T, 32, false>(p, maps, num_sms, s)
         : p.group == 64 ? launch_one<T, 64, false>(p, maps, num_sms, s)
                         : launch_one<T, 128, false>(p, maps, num_sms, s);
}

}  // namespace

cudaError_t launch_w4(const W4Params& p, int num_sms, cudaStream_t s) {
  const tc::EncodeFn f = tc::tensor_map_encoder();
  if (f == nullptr) return cudaErrorNotSupported;
  // Weights as bytes [E][N][K/2].
  Maps maps;
  const cuuint32_t one[3] = {1, 1, 1};
  const cuuint64_t size[3] = {static_cast<cuuint64_t>(p.K / 2), static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.E)};
  const cuuint64_t stride[2] = {size[0], size[0] * size[1]};
  for (int i = 0; i < 3; ++i) {
    const cuuint32_t box[3] = {kRowBytes, static_cast<cuuint32_t>((p.swiglu ? kUnitRows / 2 : kUnitRows) >> i), 1};
    if (f(&maps.box[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p.wq), size, stride, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  // Receive rows as [R][K/32][32]: a row's runs of 32 side by side, whatever
  // part of the last 256 there is.
  const cuuint64_t xsize[3] = {32, static_cast<cuuint64_t>(p.K / 32), static_cast<cuuint64_t>(p.R)};
  const cuuint64_t xstride[2] = {64, static_cast<cuuint64_t>(p.K) * 2};
  const cuuint32_t xbox[3] = {32, kSteps, 8};
  if (f(&maps.rows, p.dtype == EP_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
        const_cast<void*>(p.x), xsize, xstride, xbox, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return p.dtype == EP_DTYPE_FP16 ? launch_typed<__half>(p, maps, num_sms, s) : launch_typed<__nv_bfloat16>(p, maps, num_sms, s);
}

}  // namespace ep
