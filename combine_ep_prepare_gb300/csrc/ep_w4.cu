// ep_w4.cu -- products of a few rows per expert with 4-bit weights.
//
// w[e][n][k] = scales[e][n][k / group] * (q - 8), q the unsigned nibble k of
// row n (low nibble of a byte: even k).  out[r][n] = sum_k x[r][k] w[e][n][k]
// for the rows of expert e, or silu(gate) * up of the two halves of n.
//
// Bound by the weights' bytes.  A persistent block per SM walks units of 256,
// 128, 64 or 32 weight rows of one expert.  One warp keeps a ring of stages
// filled by TMA, running ahead across units, so that about 100 KB of weights
// per SM are in flight whatever the units' length; eight warps unpack and
// multiply.  A warp owns 32 weight rows and a share of the reduction; where
// there are few units, 2, 4 or 8 warps share 32 rows and split the reduction,
// joined through shared memory in a fixed order.
//
// The receive rows are the narrow side of mma.m16n8k16 (weights 16 x 16,
// receive rows 16 x 8): 8, 16 or 32 rows share one pass over the weights.  A
// nibble becomes 128 + q (bf16) or 1024 + q (fp16) by placing it in the
// mantissa, one packed subtraction gives q - 8 exactly, and the integers' sum
// over a group is exact up to the float32 accumulation of q x; the scale
// multiplies that sum in float32, so no weight is ever rounded.
#include <cuda.h>

#include "ep_experts.cuh"
#include "ep_tc.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;                    // consumers; one more warp loads
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kBoxRows = 32, kChunk = 128;   // a warp's weight rows and reduction elements per stage
constexpr int kBoxBytes = kBoxRows * kChunk / 2;
constexpr int kWBytes = kWarps * kBoxBytes;  // 16 KB
constexpr int kXBytes = 16 * 1024;           // row slabs of up to 8 (8 rows x kChunk) each
constexpr int kStageBytes = kWBytes + kXBytes;
constexpr int kStages = 6;

template <typename T>
struct Nib;
template <>
struct Nib<__nv_bfloat16> {
  static constexpr unsigned kMagic = 0x43004300u;   // 128
  static constexpr unsigned kOffset = 0xc308c308u;  // -136
  static __device__ __forceinline__ unsigned add(unsigned a, unsigned b) {
    unsigned r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ void mma(float* c, const unsigned* a, unsigned b0, unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Nib<__half> {
  static constexpr unsigned kMagic = 0x64006400u;   // 1024
  static constexpr unsigned kOffset = 0xe408e408u;  // -1032
  static __device__ __forceinline__ unsigned add(unsigned a, unsigned b) {
    unsigned r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ void mma(float* c, const unsigned* a, unsigned b0, unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// The eight nibbles of a word as the pairs (0,1) (2,3) (4,5) (6,7) of q - 8.
template <typename T>
__device__ __forceinline__ void unpack8(unsigned w, unsigned* out) {
  const unsigned hi = w >> 4;
#pragma unroll
  for (unsigned i = 0; i < 4; ++i) {
    const unsigned p = __byte_perm(w, hi, i | i << 4 | (4 + i) << 8 | (4 + i) << 12);
    out[i] = Nib<T>::add((p & 0x000f000fu) | Nib<T>::kMagic, Nib<T>::kOffset);
  }
}

// A unit: 256 / kw weight rows of an expert times a block of 8 nt rows.
struct Unit {
  int e, n0, r0, cnt, off, rows, nt, kw;
  bool last;  // the expert's last row block: zeroes the padding rows
};

__device__ __forceinline__ int row_tiles(int cnt) { return cnt <= 8 ? 1 : cnt <= 16 ? 2 : 4; }

struct Blocks {
  int nt, kw, nblk, tblk;
  __device__ __forceinline__ Blocks(const W4Params& p, int cnt, int KW) {
    nt = row_tiles(cnt);
    kw = KW < 8 / nt ? KW : 8 / nt;
    const int rows = kWarps * kBoxRows / kw;
    nblk = (p.N + rows - 1) / rows;  // gated: N / 2 features over rows / 2
    tblk = (cnt + 8 * nt - 1) / (8 * nt);
  }
};

struct Shared {
  uint64_t full[kStages], empty[kStages];
  int gave_up, ok, stop, kw;
  int part[32];
  int cum[EP_MAX_EXPERTS + 1];
};
constexpr int kRedBytes = 16 * 1024;
constexpr int kScaleBytes = kWarps * kBoxRows * 8 * 2;
constexpr size_t kSmemBytes = static_cast<size_t>(kStages) * kStageBytes + kRedBytes + kScaleBytes + 1024 + sizeof(Shared);

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

__device__ __forceinline__ void unit_at(const W4Params& p, const Shared& s, int u, int* e, Unit* o) {
  while (u >= s.cum[*e + 1]) ++*e;
  o->e = *e;
  o->cnt = p.counts[*e];
  o->off = p.offsets[*e];
  o->rows = p.offsets[*e + 1] - o->off;
  const Blocks b(p, o->cnt, s.kw);
  const int in = u - s.cum[*e], tb = in % b.tblk;
  o->nt = b.nt;
  o->kw = b.kw;
  o->n0 = in / b.tblk * (kWarps * kBoxRows / b.kw);
  o->r0 = tb * 8 * b.nt;
  o->last = tb + 1 == b.tblk;
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

// One unit of a consumer warp; stage and phase follow the ring.  False when a
// wait gave up.
template <typename T, int G, bool gated, int NT>
__device__ __forceinline__ bool unit_sums(const W4Params& p, const Unit& u, unsigned char* ring, T* scale_buf, Shared& s,
                                          int* stage, uint32_t* phase, float (&total)[2][NT][4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int sub = warp % u.kw, group = warp / u.kw;
  constexpr int kGroups = kChunk / G;    // scales per weight row and stage
  constexpr int kPeriod = 8 / kGroups;   // stages that eight scales of a row last
  const int ngroups = p.K / G;
  const int chunks = (p.K + kChunk - 1) / kChunk, iters = (chunks + u.kw - 1) / u.kw;
  // Box rows of this lane's fragments: fragment f's rows g and g + 8 (gated:
  // the gate row and the up row of one feature).
  int box_row[2][2];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int h = 0; h < 2; ++h) box_row[f][h] = gated ? h * 16 + f * 8 + g : f * 16 + h * 8 + g;
  // Scales: lane l brings eight of box row l, a period ahead, and the warp
  // shares them through shared memory.
  int n;  // this lane's weight row, clamped into the expert
  if (gated) {
    const int F = p.N / 2, j = u.n0 / 2 + group * 16 + (lane & 15);
    n = (j < F ? j : F - 1) + (lane >> 4) * F;
  } else {
    n = u.n0 + group * kBoxRows + lane;
    n = n < p.N ? n : p.N - 1;
  }
  const T* scale_row = static_cast<const T*>(p.scales) + (static_cast<long long>(u.e) * p.N + n) * ngroups;
  const bool wide = (ngroups & 7) == 0 && ((sub * iters * kGroups) & 7) == 0;
  auto load_scales = [&](int period) {
    const int g0 = sub * iters * kGroups + period * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (wide) {
      if (g0 < ngroups) v = __ldg(reinterpret_cast<const uint4*>(scale_row + g0));
    } else {
      unsigned short h[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        h[q] = g0 + q < ngroups ? __ldg(reinterpret_cast<const unsigned short*>(scale_row) + g0 + q) : 0;
      v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    return v;
  };
  T* scales = scale_buf + warp * (kBoxRows * 8);
  uint4 next = load_scales(0);
  float acc[2][NT][4];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) total[f][i][j] = acc[f][i][j] = 0.0f;
  bool fine = true;
  for (int it = 0; it < iters; ++it) {
    if (it % kPeriod == 0) {
      __syncwarp();
      *reinterpret_cast<uint4*>(scales + lane * 8) = next;
      __syncwarp();
      if (it + kPeriod < iters) next = load_scales(it / kPeriod + 1);
    }
    const T* sc = scales + it % kPeriod * kGroups;
    fine = __all_sync(0xffffffffu, tc::mbar_wait(tc::smem_addr(&s.full[*stage]), *phase, &s.gave_up));
    if (!fine) break;
    const unsigned char* st = ring + static_cast<size_t>(*stage) * kStageBytes;
    const unsigned char* wbox = st + warp * kBoxBytes;
    const unsigned char* xbox = st + kWBytes + sub * NT * (8 * kChunk * 2);
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint4 x[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        x[i] = *reinterpret_cast<const uint4*>(xbox + i * (8 * kChunk * 2) + kb * 512 + g * 64 + ((t ^ ((g >> 1) & 3)) << 4));
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        unsigned a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = box_row[f][h];
          unpack8<T>(*reinterpret_cast<const unsigned*>(wbox + r * 64 + ((kb ^ ((r >> 1) & 3)) << 4) + t * 4), a[h]);
        }
        const unsigned lo[4] = {a[0][0], a[1][0], a[0][1], a[1][1]}, hi[4] = {a[0][2], a[1][2], a[0][3], a[1][3]};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          Nib<T>::mma(acc[f][i], lo, x[i].x, x[i].y);
          Nib<T>::mma(acc[f][i], hi, x[i].z, x[i].w);
        }
      }
      if ((kb + 1) * 32 % G == 0) {
        const int q = kb * 32 / G;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float s0 = to_f32(sc[box_row[f][0] * 8 + q]), s1 = to_f32(sc[box_row[f][1] * 8 + q]);
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              total[f][i][j] = fmaf(j < 2 ? s0 : s1, acc[f][i][j], total[f][i][j]);
              acc[f][i][j] = 0.0f;
            }
        }
      }
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(tc::smem_addr(&s.empty[*stage]));
    if (++*stage == kStages) {
      *stage = 0;
      *phase ^= 1;
    }
  }
  return fine;
}

// Joins the reduction's shares (in ascending order) and writes the unit's output.
template <typename T, bool gated, int NT>
__device__ __forceinline__ void unit_write(const W4Params& p, const Unit& u, float* red, float (&total)[2][NT][4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int sub = warp % u.kw, group = warp / u.kw;
  if (u.kw > 1) {
    if (sub > 0) {
      float* d = red + (group * (u.kw - 1) + sub - 1) * (32 * 8 * NT);
#pragma unroll
      for (int j = 0; j < 8 * NT; ++j) d[j * 32 + lane] = total[j / (4 * NT)][j / 4 % NT][j % 4];
    }
    consumers_sync();
    if (sub > 0) return;
    for (int k = 0; k + 1 < u.kw; ++k) {
      const float* d = red + (group * (u.kw - 1) + k) * (32 * 8 * NT);
#pragma unroll
      for (int j = 0; j < 8 * NT; ++j) total[j / (4 * NT)][j / 4 % NT][j % 4] += d[j * 32 + lane];
    }
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
      for (int r = u.cnt; r < u.rows; ++r) out[static_cast<long long>(r) * cols + c] = from_f32<T>(0.0f);
  }
}

template <typename T, int G, bool gated>
__global__ void __launch_bounds__(kThreads, 1)
    ep_w4_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const W4Params p) {
  extern __shared__ unsigned char raw[];
  // Aligned by an offset, so that accesses stay known as shared-memory ones.
  unsigned char* ring = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  float* red = reinterpret_cast<float*>(ring + static_cast<size_t>(kStages) * kStageBytes);
  T* scale_buf = reinterpret_cast<T*>(ring + static_cast<size_t>(kStages) * kStageBytes + kRedBytes);
  Shared& s = *reinterpret_cast<Shared*>(ring + static_cast<size_t>(kStages) * kStageBytes + kRedBytes + kScaleBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map_w);
    tc::tma_prefetch_desc(&map_x);
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
  // The reduction is split until there are two units per block.
  const int chunks = (p.K + kChunk - 1) / kChunk;
  scan_units(p, 1, s);
  int KW = 1;
  while (KW < 8 && 2 * KW <= chunks && s.cum[p.E] * KW < 2 * static_cast<int>(gridDim.x)) KW *= 2;
  if (threadIdx.x == 0) s.kw = KW;
  __syncthreads();
  if (KW > 1) scan_units(p, KW, s);
  const int total_units = s.cum[p.E];
  int e = 0, stage = 0;
  uint32_t phase = 0;
  Unit u;
  volatile int* gave_up = &s.gave_up;
  if (warp == kWarps) {
    int issued = 0;
    for (int i = blockIdx.x; i < total_units && !*gave_up; i += gridDim.x) {
      unit_at(p, s, i, &e, &u);
      // The unit's scales into L2: the consumers read them two to eight stages ahead.
      const long long scale_bytes = static_cast<long long>(p.K / G) * 2;
      for (int r = lane; r < kWarps * kBoxRows / u.kw; r += 32) {
        const int half = kWarps * kBoxRows / u.kw / 2;
        const int n = gated ? u.n0 / 2 + (r < half ? r : p.N / 2 + r - half) : u.n0 + r;
        if (n < p.N) {
          const char* at = static_cast<const char*>(p.scales) + (static_cast<long long>(u.e) * p.N + n) * scale_bytes;
          for (long long b = 0; b < scale_bytes; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + b));
        }
      }
      const int iters = (chunks + u.kw - 1) / u.kw;
      for (int it = 0; it < iters; ++it) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(tc::smem_addr(&s.empty[stage]), phase ^ 1, gave_up))) break;
        const uint32_t full = tc::smem_addr(&s.full[stage]);
        const uint32_t w = tc::smem_addr(ring + static_cast<size_t>(stage) * kStageBytes), x = w + kWBytes;
        if (lane == 0) tc::mbar_expect(full, kWBytes + u.kw * u.nt * (8 * kChunk * 2));
        __syncwarp();
        if (lane < (gated ? 2 * kWarps : kWarps)) {
          const int cw = gated ? lane >> 1 : lane, half = gated ? lane & 1 : 0;
          const int row = gated ? half * (p.N / 2) + u.n0 / 2 + cw / u.kw * 16 : u.n0 + cw / u.kw * kBoxRows;
          tc::tma_load_3d(w + cw * kBoxBytes + half * (kBoxBytes / 2), &map_w, full, (cw % u.kw * iters + it) * (kChunk / 2),
                          row, u.e);
        }
        // A slab of 8 rows x kChunk as four boxes of 8 rows x 32 elements.
        if (lane < u.kw * u.nt * 4) {
          const int slab = lane >> 2, kb = lane & 3;
          tc::tma_load_2d(x + lane * 512, &map_x, full, (slab / u.nt * iters + it) * kChunk + kb * 32,
                          u.off + u.r0 + slab % u.nt * 8);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (*gave_up) {
      // The copies in flight land before the block's shared memory goes.
      const unsigned long long start = tc::now_ns();
      for (int j = issued < kStages ? issued : kStages; j > 0; --j) {
        if (--stage < 0) {
          stage = kStages - 1;
          phase ^= 1;
        }
        while (!tc::mbar_try(tc::smem_addr(&s.full[stage]), phase) && tc::now_ns() - start < tc::kWaitNs) {
        }
      }
      if (lane == 0) atomicOr(&p.hdr[kHdrStatus], static_cast<int>(EP_ST_TIMEOUT));
    }
  } else {
    for (int i = blockIdx.x; i < total_units; i += gridDim.x) {
      unit_at(p, s, i, &e, &u);
      bool fine;
      if (u.nt == 1) {
        float total[2][1][4];
        fine = unit_sums<T, G, gated, 1>(p, u, ring, scale_buf, s, &stage, &phase, total);
        if (fine || u.kw > 1) unit_write<T, gated, 1>(p, u, red, total);
      } else if (u.nt == 2) {
        float total[2][2][4];
        fine = unit_sums<T, G, gated, 2>(p, u, ring, scale_buf, s, &stage, &phase, total);
        if (fine || u.kw > 1) unit_write<T, gated, 2>(p, u, red, total);
      } else {
        float total[2][4][4];
        fine = unit_sums<T, G, gated, 4>(p, u, ring, scale_buf, s, &stage, &phase, total);
        if (fine || u.kw > 1) unit_write<T, gated, 4>(p, u, red, total);
      }
      if (KW > 1) {
        // All warps leave together, or the next unit's barrier would wait for one that left.
        if (threadIdx.x == 0) s.stop = *gave_up;
        consumers_sync();
        if (s.stop) break;
      } else if (!fine) {
        break;
      }
    }
  }
}

template <typename T, int G, bool gated>
cudaError_t launch_one(const W4Params& p, const CUtensorMap& w, const CUtensorMap& x, int num_sms, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(ep_w4_kernel<T, G, gated>),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(ep_w4_kernel<T, G, gated>, dim3(num_sms), dim3(kThreads), kSmemBytes, s, 0, w, x, p);
}

template <typename T>
cudaError_t launch_typed(const W4Params& p, const CUtensorMap& w, const CUtensorMap& x, int num_sms, cudaStream_t s) {
  if (p.swiglu)
    return p.group == 32   ? launch_one<T, 32, true>(p, w, x, num_sms, s)
           : p.group == 64 ? launch_one<T, 64, true>(p, w, x, num_sms, s)
                           : launch_one<T, 128, true>(p, w, x, num_sms, s);
  return p.group == 32   ? launch_one<T, 32, false>(p, w, x, num_sms, s)
         : p.group == 64 ? launch_one<T, 64, false>(p, w, x, num_sms, s)
                         : launch_one<T, 128, false>(p, w, x, num_sms, s);
}

}  // namespace

cudaError_t launch_w4(const W4Params& p, int num_sms, cudaStream_t s) {
  const tc::EncodeFn f = tc::tensor_map_encoder();
  if (f == nullptr) return cudaErrorNotSupported;
  CUtensorMap w, x;
  const cuuint32_t one[3] = {1, 1, 1};
  // weights as bytes [E][N][K/2]
  const cuuint64_t wsize[3] = {static_cast<cuuint64_t>(p.K / 2), static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.E)};
  const cuuint64_t wstride[2] = {wsize[0], wsize[0] * wsize[1]};
  const cuuint32_t wbox[3] = {kChunk / 2, static_cast<cuuint32_t>(p.swiglu ? kBoxRows / 2 : kBoxRows), 1};
  const cuuint64_t xsize[2] = {static_cast<cuuint64_t>(p.K), static_cast<cuuint64_t>(p.R)};
  const cuuint64_t xstride[1] = {static_cast<cuuint64_t>(p.K) * 2};
  const cuuint32_t xbox[2] = {32, 8};
  if (f(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p.wq), wsize, wstride, wbox, one,
        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      f(&x, p.dtype == EP_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
        const_cast<void*>(p.x), xsize, xstride, xbox, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return p.dtype == EP_DTYPE_FP16 ? launch_typed<__half>(p, w, x, num_sms, s)
                                  : launch_typed<__nv_bfloat16>(p, w, x, num_sms, s);
}

}  // namespace ep
