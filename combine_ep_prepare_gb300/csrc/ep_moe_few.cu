// ep_moe_few.cu -- a whole MoE layer for a few tokens in two kernels.
//
//   logits = x gate^T;  a = silu(g) u of w13[e] x;  out = sum_k p_k w2[e_k] a_k
//
// The first kernel takes the gate's product (and, for 8-bit weights, quantises
// the tokens).  The second is persistent, one block per SM: every block chooses
// the experts by itself, a warp a token, which costs less than handing the
// choice around; then come the gated products, one wait of the blocks for one
// another, and the down products.
//
// The chosen experts' weights are read once, so memory bounds it; everything is
// arranged to keep loads in flight and all SMs busy to the end.
// - A piece of work is 16 weight rows (8 gate rows and their 8 up rows, or 16
//   output rows of one expert) times the whole reduction; the pieces are dealt
//   out in even runs.  The 16 warps of a block split the reduction in steps of
//   128 bytes; each has its steps brought by TMA, three ahead of their use and
//   across the ends of pieces, the down products' first ones before the wait.
// - They are the 16 x K side of mma.sync as they lie: a sum does not depend on
//   its order, so 16 bytes of a row, a lane's in one load, may count as any of
//   the fragment's columns, if the tokens' operand (the same 16 bytes of token
//   lane / 4) does too.
// - Up to eight tokens of an expert, side by side, are one n-tile.  8-bit
//   weights become fp16 (exactly) on the way to the tensor cores, and the
//   tokens' 8-bit values are kept in fp16: 16 tokens, 7168 -> 2 x 2048 of 64
//   experts, took 1,056 us with mma.sync on e4m3 itself, 824 so.  A step is then
//   one block of 128, its sum scaled in float32.
// - A tile of outputs sums over experts in registers and shared memory.  Where
//   the run of a block ends inside a tile, the parts go to the workspace and
//   the block that comes last adds them in the blocks' order: no output depends
//   on which one that was.
//
// With 16-bit weights the activation is rounded to their type between the two
// products, since both operands of an mma have one type; results are then off by
// 0.0024 of their norm in bf16, 0.0016 with a float32 activation.
//
// 16-bit weights, one token: 7168 -> 2 x 2048 of 64 experts 123 us (5.7 TB/s, of
// which some 11 us are the gate, the choice and the wait); 2048 -> 2 x 1024 of
// 128 experts 33 (15 for the bytes, 9 for those three).  8-bit weights: 94 us and
// 40; 16 tokens 670 (3.4 TB/s).  Near 300 instructions a step, at 1.5 to 1.7 a
// clock, bound those: a step is half as long in bytes as it is in products, and
// no single part of it (conversion, mma, scales, tokens' words) is worth more
// than 10%.  32 tokens of 64 experts: 1,281 us in 16 bits (floor 806), 1,010 in 8
// (403), where the kernel of 17 to 32 tokens spills 304 bytes; 8 and 32 tokens,
// 2048 -> 2 x 1024 of 128 experts, 16 bits: 112 and 267 us (91 and 206).  (Times of
// calls that follow one another in a graph.)
#include <algorithm>
#include <atomic>

#include "ep_moe_few.cuh"
#include "ep_router.cuh"
#include "ep_tc.cuh"

namespace ep {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kGateThreads = 256, kGateWarps = kGateThreads / 32;
constexpr int kWarps = 16, kThreads = kWarps * 32;

constexpr int kGateTokens = 8;  // of a block

// Four e4m3 values as fp16: elements 0 and 1, 2 and 3.
__device__ __forceinline__ void fp16_of(uint32_t q, uint32_t* lo, uint32_t* hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n" : "=r"(*lo), "=r"(*hi) : "r"(q));
}
__device__ __forceinline__ uint4 fp16_of(const uint2& q) {
  uint4 r;
  fp16_of(q.x, &r.x, &r.y);
  fp16_of(q.y, &r.z, &r.w);
  return r;
}

// Block (e, y): the logits of expert e and tokens 8 y to 8 y + 7; blocks (E + t,
// 0): token t's row in 8 bits, its values kept in fp16, which holds them exactly.
template <typename G, typename T>
__global__ void __launch_bounds__(kGateThreads) ep_few_gate_kernel(const FewParams p) {
  __shared__ float part[kGateWarps][kGateTokens];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * kGateThreads + threadIdx.x; i < p.zeros; i += gridDim.x * gridDim.y * kGateThreads)
    p.hdr[i] = 0;
  if (static_cast<int>(blockIdx.x) < p.E) {
    const int e = blockIdx.x, t0 = blockIdx.y * kGateTokens;
    float acc[kGateTokens];
#pragma unroll
    for (int t = 0; t < kGateTokens; ++t) acc[t] = 0.0f;
    for (int k = threadIdx.x * 8; k < p.H; k += kGateThreads * 8) {
      Raw8<G> g;
      Raw8<T> x[kGateTokens];
      g.load(static_cast<const G*>(p.gate) + static_cast<long long>(e) * p.H + k);
#pragma unroll
      for (int t = 0; t < kGateTokens; ++t)
        if (t0 + t < p.T) x[t].load(static_cast<const T*>(p.x) + static_cast<long long>(t0 + t) * p.H + k);
      float gv[8];
      g.get(gv);
#pragma unroll
      for (int t = 0; t < kGateTokens; ++t) {
        if (t0 + t < p.T) {
          float xv[8];
          x[t].get(xv);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[t] = fmaf(gv[j], xv[j], acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kGateTokens; ++t) {
      if (t0 + t < p.T) {
        const float s = route::warp_sum(acc[t]);
        if (lane == 0) part[warp][t] = s;
      }
    }
    __syncthreads();
    if (threadIdx.x < kGateTokens && t0 + threadIdx.x < p.T) {
      float s = 0.0f;
      for (int w = 0; w < kGateWarps; ++w) s += part[w][threadIdx.x];
      p.logits[(t0 + threadIdx.x) * p.E + e] = s;
    }
  } else if (blockIdx.y == 0) {
    const int t = blockIdx.x - p.E, cols = scale_columns(p.H);
    for (int b = warp * 2; b < cols; b += kGateWarps * 2) {
      const int k = b * kF8Block + lane * 8;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (k < p.H) {
        Raw8<T> x;
        x.load(static_cast<const T*>(p.x) + static_cast<long long>(t) * p.H + k);
        x.get(v);
      }
      uint2 q;
      const float s = quantize8(v, &q);
      if (k < p.H) *reinterpret_cast<uint4*>(p.xq + static_cast<long long>(t) * p.H + k) = fp16_of(q);
      if ((lane & 15) == 0) p.xs[t * cols + b + (lane >> 4)] = k < p.H ? s : 0.0f;
    }
  }
}

// All blocks of the grid have arrived, and what they wrote before can be read.
// The word was zero when the kernel began.  False after about a second.
__device__ bool grid_wait(unsigned* word, int* status) {
  __shared__ int ok_s;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(word, 1u);
    unsigned v = 0, spins = 0;
    int ok = 1;
    for (;;) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
      if (v >= gridDim.x) break;
      if (++spins > (1u << 20)) {
        ok = 0;
        *status = static_cast<int>(EP_ST_TIMEOUT);
        break;
      }
      __nanosleep(32);
    }
    __threadfence();
    ok_s = ok;
  }
  __syncthreads();
  return ok_s != 0;
}

constexpr int kMaxRoutes = EP_MAX_FEW_TOKENS * EP_MAX_TOPK;
struct Choice {
  unsigned tokens[EP_MAX_EXPERTS];  // an expert's tokens, a bit each
  short first[EP_MAX_EXPERTS];      // the routes of the experts before it
  short used[kMaxRoutes];           // experts with a token, ascending
  short expert[kMaxRoutes];         // [t][k]
  float weight[kMaxRoutes];
  short token[kMaxRoutes];          // by expert, then token
  float share[kMaxRoutes];
  int num_used, last;
};

template <int J>
__device__ __forceinline__ void choose(const FewParams& p, Choice& c, int warp, int lane) {
  for (int t = warp; t < p.T; t += kWarps) {
    int e;
    float w;
    route::route_token<float, J>(p.router, t, lane, &e, &w);
    if (lane < p.K) {
      c.expert[t * p.K + lane] = static_cast<short>(e);
      c.weight[t * p.K + lane] = w;
      if (e >= 0) atomicOr(&c.tokens[e], 1u << t);
      if (blockIdx.x == 0) {
        p.idx[t * p.K + lane] = e;
        p.w[t * p.K + lane] = w;
      }
    }
  }
}

// The choice, and the routes sorted by expert.
__device__ __forceinline__ void choose_experts(const FewParams& p, Choice& c, int warp, int lane) {
  for (int e = threadIdx.x; e < p.E; e += kThreads) c.tokens[e] = 0;
  __syncthreads();
  const int j = (p.E + 31) / 32;
  if (j <= 2) choose<2>(p, c, warp, lane);
  else if (j <= 4) choose<4>(p, c, warp, lane);
  else if (j <= 8) choose<8>(p, c, warp, lane);
  else choose<32>(p, c, warp, lane);
  __syncthreads();
  if (warp == 0) {
    int used = 0, first = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < p.E ? __popc(c.tokens[e]) : 0;
      int sum = n;
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, sum, d);
        if (lane >= d) sum += o;
      }
      const unsigned has = __ballot_sync(kAll, n > 0);
      if (n > 0) {
        c.used[used + __popc(has & ((1u << lane) - 1))] = static_cast<short>(e);
        c.first[e] = static_cast<short>(first + sum - n);
      }
      used += __popc(has);
      first += __shfl_sync(kAll, sum, 31);
    }
    if (lane == 0) c.num_used = used;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < p.T * p.K; r += kThreads) {
    const int t = r / p.K, e = c.expert[r];
    if (e < 0) continue;
    const int at = c.first[e] + __popc(c.tokens[e] & ((1u << t) - 1));
    c.token[at] = static_cast<short>(t);
    c.share[at] = c.weight[r];
  }
  __syncthreads();
}

// One box of weights to this block's shared memory.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, uint32_t bar, bool down, int x, int row, int e) {
  if (down)
    tc::tma_load_3d(dst, m, bar, x, row, e);
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(x), "r"(row), "r"(0), "r"(e)
        : "memory");
}

// d += a b: a the 16 weight rows' words, b the 8 tokens'.
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Where a piece of work lies: its expert, its two eights of weight rows and the
// rows of the tokens' operand.
struct Piece {
  int u, e;                   // its place among the used experts, its number
  int row0, row1, n, pos;     // rows of the expert's matrix (row1 < 0: none); tokens, and the first one's route
  int tile;                   // features (gate and up) or outputs, from 8 tile or 16 tile on
};

// One of the two products' pieces, in the order in which they are dealt out.
template <bool down>
struct Walk {
  const FewParams& p;
  const Choice& c;
  int tiles, u, tile;  // up: by expert, then tile; down: by tile, then expert
  __device__ __forceinline__ Walk(const FewParams& p_, const Choice& c_, int i) : p(p_), c(c_) {
    tiles = down ? (p.H + kFewRows - 1) / kFewRows : p.F / 8;
    u = down ? i % max(1, c.num_used) : i / tiles;
    tile = down ? i / max(1, c.num_used) : i % tiles;
  }
  __device__ __forceinline__ void advance(int by) {
    if (down) {
      for (u += by; u >= c.num_used; u -= c.num_used) ++tile;
    } else {
      for (tile += by; tile >= tiles; tile -= tiles) ++u;
    }
  }
  __device__ __forceinline__ Piece at() const {
    Piece o;
    o.u = u;
    o.e = c.used[u];
    o.n = __popc(c.tokens[o.e]);
    o.pos = c.first[o.e];
    o.tile = tile;
    if (down) {
      o.row0 = tile * kFewRows;
      o.row1 = o.row0 + 8 < p.H ? o.row0 + 8 : -1;
    } else {
      o.row0 = tile * 8;
      o.row1 = p.F + o.row0;
    }
    return o;
  }
};

// Steps of weights in flight: boxes of 16 rows x 128 bytes that a warp's first
// lane has brought to the warp's own slots of shared memory.  (Loads by the
// lanes themselves touch eight lines each, 64 bytes of them; two or three steps
// of them in registers took 127 and 104 us for one token, 7168 -> 2 x 2048, in
// 16 and in 8 bits, cp.async 157 and 130.)
constexpr int kAhead = 3, kStepBytes = 128, kSlotBytes = kFewRows * kStepBytes;
constexpr int kRingBytes = kWarps * kAhead * kSlotBytes;
struct Ring {
  uint32_t data, full;  // this warp's slots and their barriers
  volatile int* gave_up;
  int slot;
  uint32_t phase;
  __device__ __forceinline__ void next() {
    if (++slot == kAhead) {
      slot = 0;
      phase ^= 1;
    }
  }
};
__device__ __forceinline__ float load_shared(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
// The place in a box of the fragment's row g: rows of neighbouring lanes differ
// in the bit that makes the 128-byte swizzle swap a row's halves, so that a
// warp's 16-byte loads meet all banks.
__device__ __forceinline__ int box_row(int g) { return (g >> 1) | (g & 1) << 2; }

// How many steps of the tokens' operand are in registers at a time (with one, it
// comes half a step at a time, just before its use), and the pieces of the gated
// products that are joined at a time.
template <bool f8, int NT>
struct Depth {
  static constexpr int kTokens = NT == 1 || (NT == 2 && !f8) ? 2 : 1;
  static constexpr int kBatch = 4 / NT;
};
constexpr int kRedFloats = 2 * 4 * kWarps * 16 * 8;  // two batches' sums

// How a block's warps share its run: groups of them take a piece each in turn,
// and split its reduction among them.
struct Team {
  int groups, group, split, sub;  // groups, this warp's; warps of a group, this one's place
  __device__ __forceinline__ Team(int pieces, int steps, int warp) {
    // A piece costs a warp as much as a step or two beside its steps, so groups
    // with more steps of fewer pieces are faster (7168 -> 2 x 2048 in 8 bits: 16
    // tokens of 64 experts 717 us with one group, 672 with this rule; 32 tokens
    // 1,331 and 1,010; 32 experts in 16 bits 720 and 621).  With few pieces the
    // groups would not come out even (one token in 16 bits: 125 us with one,
    // 128 where the rule asks for half as many pieces).
    groups = 1;
    while (groups < 4 && pieces >= 16 * groups && (steps * groups + kWarps - 1) / kWarps < 8) groups *= 2;
    split = kWarps / groups;
    group = warp / split;
    sub = warp % split;
  }
};

// A block's run [lo, hi) of pieces: of each of its group's pieces, warp w of
// the group takes the steps w, w + split, ... of the reduction (128 bytes of a
// row each).  put(piece, its place in the segment, sums) is called when a
// piece's steps are over, join(segment) by all warps when a segment's pieces
// are; wait() when the weights' first steps are on their way.
template <typename T, bool f8, int NT, bool down, typename Done>
__device__ __forceinline__ void run_pieces(const FewParams& p, const Choice& c, const CUtensorMap& map, Ring& ring, int lo, int hi, const Team& team,
                                           int lane, Done done) {
  using E = typename std::conditional<f8, uint8_t, T>::type;
  constexpr int kWords = f8 ? 4 : 2;  // 16-byte words of a token that meet a lane's two of a weight row
  constexpr int kTokens = Depth<f8, NT>::kTokens;
  constexpr bool ahead = kTokens > 1;
  const int red = (down ? p.F : p.H) * static_cast<int>(sizeof(E)), rows = down ? p.H : 2 * p.F;  // red in bytes
  const int turns = ((red + kStepBytes - 1) / kStepBytes + team.split - 1) / team.split, stride = team.split * kStepBytes;
  const int own = max(0, (hi - lo - team.group + team.groups - 1) / team.groups), total = own * turns;
  const int g = lane >> 2, t = lane & 3;
  const int k0 = team.sub * kStepBytes + t * 16;  // this lane's first byte of a row
  const char* x = f8 ? reinterpret_cast<const char*>(down ? p.aq : p.xq) : static_cast<const char*>(down ? p.act : p.x);
  const uint32_t scales = done.token_scales();
  const int xcols = f8 ? scale_columns(red) : 0, wcols = f8 ? f8_blocks(red) : 0, wblocks = f8 ? f8_blocks(rows) : 0;
  const uint32_t in_box = box_row(g) * kStepBytes + ((t ^ box_row(g)) & 7) * 16;  // the lane's first word; the other half's: bit 6 the other way
  uint4 b[kTokens][NT][ahead ? kWords : kWords / 2];
  float sw[kTokens][2], sx[kTokens][NT][2];
  // The weights' place.
  struct {
    int row, e, turn;
  } at_a;
  // The tokens': byte offsets of their rows and of their scales' rows.  Columns
  // past the last token repeat it: nothing reads their sums.
  struct {
    int row[NT], scale[NT][2], turn, n;
    const float *w0, *w1;
  } at_b;
  Walk<down> walk_a(p, c, lo + team.group), walk_b(walk_a), walk_c(walk_a);
  auto place_a = [&]() {
    const Piece o = walk_a.at();
    at_a.row = o.row0;
    at_a.e = o.e;
    at_a.turn = 0;
  };
  auto place_b = [&]() {
    const Piece o = walk_b.at();
    at_b.turn = 0;
    at_b.n = o.n;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int col = min(8 * i + g, o.n - 1);
      at_b.row[i] = ((down ? o.pos + col : c.token[o.pos + col]) * red + k0) * (f8 ? 2 : 1);
      if constexpr (f8) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int col2 = min(8 * i + 2 * t + q, o.n - 1);
          at_b.scale[i][q] = (down ? o.pos + col2 : c.token[o.pos + col2]) * xcols;
        }
      }
    }
    if constexpr (f8) {
      const float* s = p.s13;
      if (down) s = p.s2;
      at_b.w0 = s + (static_cast<long long>(o.e) * wblocks + o.row0 / kF8Block) * wcols;
      at_b.w1 = down ? at_b.w0 : s + (static_cast<long long>(o.e) * wblocks + o.row1 / kF8Block) * wcols;
    }
  };
  // By the first lane alone; what lies past a row's or the matrix's end comes as zeros.
  auto load_a = [&](int slot) {
    const uint32_t bar = ring.full + 8 * slot;
    tc::mbar_expect(bar, kSlotBytes);
    load_box(ring.data + slot * kSlotBytes, &map, bar, down, team.sub * kStepBytes + at_a.turn * stride, at_a.row, at_a.e);
    if (++at_a.turn == turns) {
      walk_a.advance(team.groups);
      if (walk_a.u < c.num_used && walk_a.tile < walk_a.tiles) place_a();
    }
  };
  // Words [from, from + count) of the step's tokens' operand.
  auto load_words = [&](int to, int from, int count) {
    const int k = at_b.turn * stride;
    // Word j of what is asked for, in 16-byte words from the lane's first on.
    auto word = [&](int j) { return 4 * ((from + j) / (kWords / 2)) * (kWords / 2) + (from + j) % (kWords / 2); };
    if (k + (team.sub + 1) * kStepBytes <= red) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (NT > 1 && 8 * i >= at_b.n) break;
        const uint4* row = reinterpret_cast<const uint4*>(x + at_b.row[i] + k * (f8 ? 2 : 1));
#pragma unroll
        for (int j = 0; j < kWords; ++j)  // act is written in this kernel: not through the read-only path
          if (j < count) b[to][i][j] = down ? __ldcg(row + word(j)) : __ldg(row + word(j));
      }
    } else {  // the row's end: zeros past it
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (NT > 1 && 8 * i >= at_b.n) break;
        const uint4* row = reinterpret_cast<const uint4*>(x + at_b.row[i] + k * (f8 ? 2 : 1));
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          if (j >= count) break;
          b[to][i][j] = make_uint4(0, 0, 0, 0);
          if (k + k0 + 64 * ((from + j) / (kWords / 2)) < red) b[to][i][j] = down ? __ldcg(row + word(j)) : __ldg(row + word(j));
        }
      }
    }
  };
  // The step's scales, and on to the next.
  auto load_scales = [&](int to) {
    if constexpr (f8) {
      // One block of 128 a step.  A step past the end has zeros, times the last block's scale.
      const int block = min(team.sub + at_b.turn * team.split, wcols - 1);
      sw[to][0] = __ldg(at_b.w0 + block);
      sw[to][1] = down ? sw[to][0] : __ldg(at_b.w1 + block);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          sx[to][i][q] = down ? __ldcg(p.as + at_b.scale[i][q] + block) : load_shared(scales + 4 * (at_b.scale[i][q] + block));
    }
  };
  auto next_b = [&]() {
    if (++at_b.turn == turns) {
      walk_b.advance(team.groups);
      if (walk_b.u < c.num_used && walk_b.tile < walk_b.tiles) place_b();
    }
  };
  auto load_b = [&](int to) {
    load_words(to, 0, kWords);
    load_scales(to);
    next_b();
  };
  if (total > 0) place_a();
  if (lane == 0)
    for (int q = 0, slot = ring.slot; q < min(kAhead, total); ++q) {
      load_a(slot);
      slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
  done.wait();
  if (total > 0) place_b();
  if (ahead && total > 0) load_b(1);
  float sum[NT][4];
  int n = 0, n_tokens = 0;
  auto step = [&]() {
    if constexpr (ahead) {
      // The words change places, not the code: a copy of a step for each buffer
      // of them misses the instruction cache (one token, 7168 -> 2 x 2048: 123 us
      // with one copy, 126 with two, 134 with four).
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) b[0][i][j] = b[1][i][j];
        if constexpr (f8) {
          sx[0][i][0] = sx[1][i][0];
          sx[0][i][1] = sx[1][i][1];
        }
      }
      if constexpr (f8) {
        sw[0][0] = sw[1][0];
        sw[0][1] = sw[1][1];
      }
      if (n + 1 < total) load_b(1);
    } else {
      load_scales(0);
    }
    tc::mbar_wait(ring.full + 8 * ring.slot, ring.phase, ring.gave_up);
    const uint32_t in = ring.data + ring.slot * kSlotBytes + in_box;
    float d[NT][4] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!ahead) load_words(0, h * kWords / 2, kWords / 2);
      uint32_t u[4], v[4];
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(in ^ (h * 64)) : "memory");
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"((in ^ (h * 64)) + 1024) : "memory");
#pragma unroll
      for (int j = 0; j < (f8 ? 4 : 2); ++j) {
        uint32_t u0 = u[2 * j & 3], u1 = u[(2 * j + 1) & 3], v0 = v[2 * j & 3], v1 = v[(2 * j + 1) & 3];
        if constexpr (f8) {
          fp16_of(u[j], &u0, &u1);
          fp16_of(v[j], &v0, &v1);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if (NT > 1 && 8 * i >= n_tokens) break;
          const uint4& y = b[0][i][(ahead ? h * kWords / 2 : 0) + j / 2];
          mma<typename std::conditional<f8, __half, T>::type>(f8 ? d[i] : sum[i], u0, v0, u1, v1, j & 1 ? y.z : y.x, j & 1 ? y.w : y.y);
        }
      }
    }
    __syncwarp();  // read by all lanes: the slot may be written again
    if (n + kAhead < total && lane == 0) load_a(ring.slot);
    ring.next();
    if constexpr (f8) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(d[i][j], sw[0][j >> 1] * sx[0][i][j & 1], sum[i][j]);
    }
    if (!ahead) next_b();
    ++n;
  };
  int mine = lo + team.group;
  for (int first = lo; first < hi;) {
    const int stop = done.segment_end(first, hi);
    for (; mine < stop; mine += team.groups) {
      const Piece o = walk_c.at();
      n_tokens = o.n;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = 0.0f;
#pragma unroll 1
      for (int turn = 0; turn < turns; ++turn) step();
      done.put(o, mine - first, sum);
      walk_c.advance(team.groups);
    }
    done.join(first, stop, stop == hi);
    first = stop;
  }
}

// After a piece of the gated products its warps' sums go to shared memory;
// after kBatch pieces of each group they are joined and the activation is taken
// and written; with 8-bit weights it is quantised at the end of the run.
template <typename T, bool f8, int NT>
struct UpDone {
  static constexpr int kCols = 8 * NT, kBatch = Depth<f8, NT>::kBatch;
  static constexpr int kWarpFloats = 16 * kCols;
  static_assert(2 * kBatch * kWarps * kWarpFloats == kRedFloats, "shared memory");
  const FewParams& p;
  Choice& c;
  float* red;  // [2][kBatch pieces of each group][its warps][16][kCols]
  const Team& team;
  int warp, lane, lo, turn;
  uint32_t scales;  // 8-bit weights: the tokens', in shared memory
  __device__ __forceinline__ uint32_t token_scales() const { return scales; }
  __device__ __forceinline__ void wait() const {}
  __device__ __forceinline__ int segment_end(int first, int hi) const { return min(hi, first + kBatch * team.groups); }
  __device__ __forceinline__ void put(const Piece& o, int b, const float (&sum)[NT][4]) const {
    float* mine = red + (turn * kBatch * kWarps + b * team.split + team.sub) * kWarpFloats;
    const int g = box_row(lane >> 2), t = lane & 3;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (8 * i >= o.n) break;
      *reinterpret_cast<float2*>(mine + g * kCols + 8 * i + 2 * t) = make_float2(sum[i][0], sum[i][1]);
      *reinterpret_cast<float2*>(mine + (g + 8) * kCols + 8 * i + 2 * t) = make_float2(sum[i][2], sum[i][3]);
    }
  }
  __device__ __forceinline__ void join(int first, int stop, bool end) {
    __syncthreads();
    for (int j = threadIdx.x; j < (stop - first) * 8 * kCols; j += kThreads) {
      const int col = j % kCols, f = j / kCols % 8, b = j / (8 * kCols);
      const Piece q = Walk<false>(p, c, first + b).at();
      if (col < q.n) {
        const float* at = red + (turn * kBatch * kWarps + b * team.split) * kWarpFloats + f * kCols + col;
        float gate = 0.0f, up = 0.0f;
#pragma unroll 4
        for (int w = 0; w < team.split; ++w) {
          gate += at[w * kWarpFloats];
          up += at[w * kWarpFloats + 8 * kCols];
        }
        const float a = swiglu(gate, up);
        const long long i = static_cast<long long>(q.pos + col) * p.F + q.tile * 8 + f;
        if constexpr (f8) static_cast<float*>(p.act)[i] = a;
        else static_cast<T*>(p.act)[i] = from_f32<T>(a);
      }
    }
    turn ^= 1;  // the other buffer next: the sums here are still being read
    if constexpr (f8)
      if (end) quantize_run(stop);
  }
  // The run's features to 8 bits, a block of 128 (16 pieces) at a time.  The
  // first and the last may be other blocks' too: who brings the last piece
  // quantises them.
  __device__ __forceinline__ void quantize_run(int hi) const {
    constexpr int kPieces = kF8Block / 8;
    const int b0 = lo / kPieces, b1 = (hi - 1) / kPieces;
    __threadfence();
    if (threadIdx.x == 0) c.last = 0;
    __syncthreads();
    if (threadIdx.x < 2 && (threadIdx.x == 0 || b1 != b0)) {
      const int b = threadIdx.x == 0 ? b0 : b1;
      const int mine = min(hi, (b + 1) * kPieces) - max(lo, b * kPieces);
      if (mine == kPieces || atomicAdd(p.written + b, mine) + mine == kPieces) atomicOr(&c.last, 1 << threadIdx.x);
      __threadfence();
    }
    __syncthreads();
    for (int b = b0; b <= b1; ++b) {
      if (b == b0 ? c.last & 1 : b < b1 || (c.last & 2)) quantize(Walk<false>(p, c, b * kPieces).at());
    }
  }
  __device__ __forceinline__ void quantize(const Piece& o) const {
    const int block = o.tile / (kF8Block / 8);
    for (int col = warp; col < o.n; col += kWarps) {
      const long long at = static_cast<long long>(o.pos + col) * p.F + block * kF8Block + lane * 4;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(p.act) + at));
      float m = max_nan(max_nan(fabsf(v.x), fabsf(v.y)), max_nan(fabsf(v.z), fabsf(v.w)));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, d));
      const BlockScale s = block_scale(m);
      uint2 q;
      fp16_of(e4m3x4(v.x * s.inv, v.y * s.inv, v.z * s.inv, v.w * s.inv), &q.x, &q.y);
      *reinterpret_cast<uint2*>(p.aq + at) = q;
      if (lane == 0) p.as[static_cast<long long>(o.pos + col) * scale_columns(p.F) + block] = s.scale;
    }
  }
};

// After a piece of the down products: its sums, times the tokens' shares, are
// added to this warp's sums of the tile; after the tile's last piece here the
// warps' sums are joined.
template <typename T, int NT>
struct DownDone {
  const FewParams& p;
  Choice& c;
  float* red;  // [kWarps][16][T]
  int warp, lane, lo, pieces, blocks;  // blocks: those that have pieces
  __device__ __forceinline__ uint32_t token_scales() const { return 0; }
  __device__ __forceinline__ void zero() const {
    for (int i = lane; i < 16 * p.T; i += 32) red[warp * 16 * p.T + i] = 0.0f;
    __syncwarp();
  }
  __device__ __forceinline__ void wait() const {
    grid_wait(reinterpret_cast<unsigned*>(p.hdr + 1), p.hdr);  // given up: the sums are of what happens to be in act
    zero();
  }
  __device__ __forceinline__ int block_of(long long piece) const {
    return static_cast<int>(((piece + 1) * blocks - 1) / pieces);
  }
  __device__ __forceinline__ int start_of(long long block) const { return static_cast<int>(block * pieces / blocks); }
  __device__ __forceinline__ int segment_end(int first, int hi) const { return min(hi, (first / c.num_used + 1) * c.num_used); }
  __device__ __forceinline__ void put(const Piece& o, int, const float (&sum)[NT][4]) const {
    float* mine = red + warp * 16 * p.T;
    const int g = box_row(lane >> 2), t = lane & 3;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (8 * i >= o.n) break;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int col = 8 * i + 2 * t + q;
        if (col < o.n) {
          const int token = c.token[o.pos + col];
          const float share = c.share[o.pos + col];
          mine[g * p.T + token] = fmaf(share, sum[i][q], mine[g * p.T + token]);
          mine[(g + 8) * p.T + token] = fmaf(share, sum[i][2 + q], mine[(g + 8) * p.T + token]);
        }
      }
    }
    __syncwarp();  // an expert's columns are other lanes' in the next piece
  }
  __device__ __forceinline__ void join(int first, int, bool end) const {
    const int at = first / c.num_used;  // the tile
    __syncthreads();
    const bool alone = first_block(at) == last_block(at);
    for (int i = threadIdx.x; i < 16 * p.T; i += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[w * 16 * p.T + i];
      if (alone) store(at, i, s);
      else part_of(blockIdx.x, at)[i] = s;
    }
    if (end) {
      // This block's first and last tile may be others' too: it says that its
      // parts are there, and adds up the tiles of which it is the last to say so.
      const int begins = lo / c.num_used;
      __threadfence();
      if (threadIdx.x == 0) c.last = 0;
      __syncthreads();
      if (threadIdx.x < 2) {
        const int tile = threadIdx.x == 0 ? begins : at, others = last_block(tile) - first_block(tile);
        if (others > 0 && (threadIdx.x == 0 || tile != begins) && atomicAdd(p.done + tile, 1) == others) atomicOr(&c.last, 1 << threadIdx.x);
        __threadfence();
      }
      __syncthreads();
      for (int left = c.last; left; left &= left - 1) {
        const int tile = left & 1 ? begins : at;
        for (int i = threadIdx.x; i < 16 * p.T; i += kThreads) {
          float s = 0.0f;
          for (int b = first_block(tile); b <= last_block(tile); ++b) s += __ldcg(part_of(b, tile) + i);
          store(tile, i, s);
        }
      }
      return;
    }
    __syncthreads();  // read: the sums begin again
    zero();
  }
  __device__ __forceinline__ int first_block(int tile) const { return block_of(static_cast<long long>(tile) * c.num_used); }
  __device__ __forceinline__ int last_block(int tile) const { return block_of(static_cast<long long>(tile + 1) * c.num_used - 1); }
  // A block has a place for its first tile's part and one for its last tile's.
  __device__ __forceinline__ float* part_of(int block, int tile) const {
    return p.part + (static_cast<long long>(block) * 2 + (start_of(block) / c.num_used == tile ? 0 : 1)) * 16 * p.T;
  }
  __device__ __forceinline__ void store(int tile, int i, float s) const {
    const int h = tile * kFewRows + i / p.T;
    if (h < p.H) static_cast<T*>(p.out)[static_cast<long long>(i % p.T) * p.H + h] = from_f32<T>(s);
  }
};

// This block's even share of the pieces; where there are fewer than blocks, the
// last blocks have none.
struct Run {
  int pieces, blocks, lo, hi;
  __device__ __forceinline__ explicit Run(long long n) : pieces(static_cast<int>(n)), blocks(static_cast<int>(min(n, static_cast<long long>(gridDim.x)))) {
    const long long b = min(static_cast<int>(blockIdx.x), blocks);
    lo = static_cast<int>(b * n / blocks);
    hi = static_cast<int>(min(b + 1, static_cast<long long>(blocks)) * n / blocks);
  }
};

template <typename T, bool f8, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    ep_few_experts_kernel(const __grid_constant__ CUtensorMap map13, const __grid_constant__ CUtensorMap map2, const FewParams p) {
  __shared__ Choice c;
  __shared__ uint64_t full[kWarps * kAhead];
  __shared__ int gave_up;
  extern __shared__ unsigned char raw[];
  unsigned char* memory = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  float* red = reinterpret_cast<float*>(memory + kRingBytes);
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map13);
    tc::tma_prefetch_desc(&map2);
    for (int i = 0; i < kWarps * kAhead; ++i) tc::mbar_init(tc::smem_addr(&full[i]), 1);
    tc::mbar_init_fence();
    gave_up = 0;
  }
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Ring ring{tc::smem_addr(memory) + warp * (kAhead * kSlotBytes), tc::smem_addr(&full[warp * kAhead]), &gave_up, 0, 0};
  float* scales = red + kRedFloats;
  if constexpr (f8)
    for (int i = threadIdx.x; i < p.T * scale_columns(p.H); i += kThreads) scales[i] = p.xs[i];
  choose_experts(p, c, warp, lane);  // has barriers
  if (c.num_used == 0) {
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < static_cast<long long>(p.T) * p.H; i += static_cast<long long>(gridDim.x) * kThreads)
      static_cast<T*>(p.out)[i] = from_f32<T>(0.0f);
    return;
  }
  constexpr int es = f8 ? 1 : 2;
  {
    const Run run(static_cast<long long>(c.num_used) * (p.F / 8));
    const Team team(run.pieces / run.blocks, (p.H * es + kStepBytes - 1) / kStepBytes, warp);
    run_pieces<T, f8, NT, false>(p, c, map13, ring, run.lo, run.hi, team, lane,
                                 UpDone<T, f8, NT>{p, c, red, team, warp, lane, run.lo, 0, tc::smem_addr(scales)});
  }
  {
    const Run run(static_cast<long long>(c.num_used) * ((p.H + kFewRows - 1) / kFewRows));
    const Team team(run.pieces / run.blocks, (p.F * es + kStepBytes - 1) / kStepBytes, warp);
    run_pieces<T, f8, NT, true>(p, c, map2, ring, run.lo, run.hi, team, lane,
                                DownDone<T, NT>{p, c, red, warp, lane, run.lo, run.pieces, run.blocks});
  }
  __syncthreads();
  if (threadIdx.x == 0 && gave_up) {
    *p.hdr = static_cast<int>(EP_ST_TIMEOUT);
    // Copies in flight land before the block's shared memory goes; one takes microseconds.
    const unsigned long long start = tc::now_ns();
    while (tc::now_ns() - start < tc::kWaitNs / 100) {
    }
  }
}

// A map of [dim 3]..[dim 1][dim 0] bytes, strides of the dimensions from 1 on.
bool byte_map(CUtensorMap* m, const void* base, int dims, const long long (&size)[4], const long long (&stride)[3], const int (&box)[4]) {
  const tc::EncodeFn f = tc::tensor_map_encoder();
  if (f == nullptr) return false;
  cuuint64_t sz[4], st[3];
  cuuint32_t bx[4];
  const cuuint32_t one[4] = {1, 1, 1, 1};
  for (int i = 0; i < dims; ++i) {
    sz[i] = static_cast<cuuint64_t>(size[i]);
    bx[i] = static_cast<cuuint32_t>(box[i]);
    if (i + 1 < dims) st[i] = static_cast<cuuint64_t>(stride[i]);
  }
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(dims), const_cast<void*>(base), sz, st, bx, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The second kernel's blocks: one per SM that can hold one, all at once.
template <typename T, bool f8, int NT>
cudaError_t launch_experts(const FewParams& p, int num_sms, cudaStream_t s) {
  constexpr size_t most = 1024 + kRingBytes + sizeof(float) * (kRedFloats + (f8 ? 8 * NT * (EP_MAX_NORM_HIDDEN / kF8Block) : 0));
  const size_t smem = 1024 + kRingBytes + sizeof(float) * (kRedFloats + (f8 ? p.T * scale_columns(p.H) : 0));
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  const auto kern = ep_few_experts_kernel<T, f8, NT>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int blocks = known[dev].load(std::memory_order_acquire);
  if (blocks == 0) {
    int per_sm = 0;
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, most);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorLaunchOutOfResources;
    blocks = std::min(num_sms, kFewBlocksMax);
    known[dev].store(blocks, std::memory_order_release);
  }
  const long long es = f8 ? 1 : 2, h = p.H * es, f = p.F * es;  // rows in bytes
  CUtensorMap map13, map2;
  if (!byte_map(&map13, p.w13, 4, {h, p.F, 2, p.E}, {h, h * p.F, h * 2 * p.F}, {kStepBytes, 8, 2, 1}) ||
      !byte_map(&map2, p.w2, 3, {f, p.H, p.E, 1}, {f, f * p.H, 0}, {kStepBytes, kFewRows, 1, 1}))
    return cudaErrorInvalidValue;
  return launch_pdl_ex(kern, dim3(blocks), dim3(kThreads), smem, s, 0, true, map13, map2, p);
}

template <typename T, bool f8>
cudaError_t launch_sized(const FewParams& p, int num_sms, cudaStream_t s) {
  if (p.T <= 8) return launch_experts<T, f8, 1>(p, num_sms, s);
  if (p.T <= 16) return launch_experts<T, f8, 2>(p, num_sms, s);
  return launch_experts<T, f8, 4>(p, num_sms, s);
}

template <typename T>
cudaError_t launch_typed(const FewParams& p, int num_sms, cudaStream_t s) {
  const dim3 grid(p.E + (p.f8 ? p.T : 0), (p.T + kGateTokens - 1) / kGateTokens), block(kGateThreads);
  const cudaError_t e = p.gate_dtype == EP_DTYPE_FP32   ? launch_pdl(ep_few_gate_kernel<float, T>, grid, block, 0, s, 0, p)
                        : p.gate_dtype == EP_DTYPE_FP16 ? launch_pdl(ep_few_gate_kernel<__half, T>, grid, block, 0, s, 0, p)
                                                        : launch_pdl(ep_few_gate_kernel<__nv_bfloat16, T>, grid, block, 0, s, 0, p);
  if (e != cudaSuccess) return e;
  return p.f8 ? launch_sized<T, true>(p, num_sms, s) : launch_sized<T, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_moe_few(const FewParams& p, int num_sms, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP16) return launch_typed<__half>(p, num_sms, s);
  return launch_typed<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace ep
