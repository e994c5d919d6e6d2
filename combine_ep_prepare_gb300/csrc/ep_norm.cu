// ep_norm.cu -- root-mean-square norm with the residual's addition and an
// 8-bit output, its gradient, and the quantisation of rows.
//
//   h = round(x + residual),  r = (mean h^2 + eps)^-1/2,  y = h r w
//   dh = dsum + r (w dy - h r^2 c),  c = mean(w dy h);  dw = sum_t dy h r
//
// All are bound by memory: a row is read once into registers, eight elements
// (16 bytes of a 16-bit type) a thread and step, and everything is computed
// from there.  Sixteen lanes then hold a block of 128, so that its largest
// magnitude is four shuffles.
#include <algorithm>

#include "ep_f8.cuh"

namespace ep {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// Sums of a and b over the block's threads, in every thread; `part` holds 64
// floats that no thread still reads.
__device__ __forceinline__ float2 block_sum2(float a, float b, float* part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    a += __shfl_xor_sync(kAll, a, d);
    b += __shfl_xor_sync(kAll, b, d);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return make_float2(a, b);
  if (lane == 0) {
    part[2 * warp] = a;
    part[2 * warp + 1] = b;
  }
  __syncthreads();
  a = lane < warps ? part[2 * lane] : 0.0f;
  b = lane < warps ? part[2 * lane + 1] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    a += __shfl_xor_sync(kAll, a, d);
    b += __shfl_xor_sync(kAll, b, d);
  }
  return make_float2(a, b);
}

// One block per row; thread t has the vectors t, t + blockDim, ...
template <typename T, int NV>
__global__ void __launch_bounds__(1024) ep_norm_kernel(const NormParams p) {
  __shared__ float part[64];
  pdl_wait();
  const int vectors = p.H / 8;
  const long long row = static_cast<long long>(blockIdx.x) * p.H;
  const T* x = static_cast<const T*>(p.x) + row;
  const T* res = p.residual != nullptr ? static_cast<const T*>(p.residual) + row : nullptr;
  float h[NV][8], ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
    if (v < vectors) {
      Raw8<T> a;
      a.load_rw(x + 8 * v);
      a.get(h[i]);
      if (res != nullptr) {
        Raw8<T> b;
        float r[8];
        b.load_rw(res + 8 * v);
        b.get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = to_f32(from_f32<T>(h[i][j] + r[j]));
        if (p.sum != nullptr) store8<T>(static_cast<T*>(p.sum) + row + 8 * v, h[i]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
  }
  ss = block_sum2(ss, 0.0f, part).x;
  const float r = 1.0f / sqrtf(ss / static_cast<float>(p.H) + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < vectors) {
      Raw8<T> a;
      float w[8];
      a.load(static_cast<const T*>(p.weight) + 8 * v);
      a.get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * r * w[j];
      if (p.y != nullptr) store8<T>(static_cast<T*>(p.y) + row + 8 * v, h[i]);
    }
    if (p.q != nullptr) {
      uint2 q;
      const float s = quantize8(h[i], &q);
      if (v < vectors) {
        *reinterpret_cast<uint2*>(p.q + row + 8 * v) = q;
        if ((v & 15) == 0) p.scales[static_cast<long long>(blockIdx.x) * scale_columns(p.H) + v / 16] = s;
      }
    }
  }
  if (p.q != nullptr)
    for (int b = f8_blocks(p.H) + threadIdx.x; b < scale_columns(p.H); b += blockDim.x)
      p.scales[static_cast<long long>(blockIdx.x) * scale_columns(p.H) + b] = 0.0f;
}

// A thread's vector of a row's gradients and h.
template <typename T>
struct GradVec {
  Raw8<T> dy, h, ds;
  __device__ __forceinline__ void load(const NormParams& p, unsigned t, int v, bool stream) {
    const long long at = static_cast<long long>(t) * p.H + 8 * v;
    dy.load_rw(static_cast<const T*>(p.dy) + at);
    h.load_rw(static_cast<const T*>(p.x) + at);
    if (stream && p.dsum != nullptr) ds.load_rw(static_cast<const T*>(p.dsum) + at);
  }
  __device__ __forceinline__ void sums(const float (&w)[8], float* ss, float* inner) const {
    float a[8], b[8];
    dy.get(a);
    h.get(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      *ss = fmaf(b[j], b[j], *ss);
      *inner = fmaf(a[j] * w[j], b[j], *inner);
    }
  }
  __device__ __forceinline__ void finish(const NormParams& p, unsigned t, int v, const float (&w)[8], float r, float c, float (&dw)[8]) const {
    float a[8], b[8], s[8];
    dy.get(a);
    h.get(b);
    if (p.dsum != nullptr) {
      ds.get(s);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] = fmaf(a[j] * r, b[j], dw[j]);
      s[j] = fmaf(r, fmaf(-b[j], c, a[j] * w[j]), s[j]);
    }
    store8<T>(static_cast<T*>(p.dh) + static_cast<long long>(t) * p.H + 8 * v, s);
  }
};

// Blocks stride over the rows; a thread keeps its columns' share of dw.  One
// vector a thread (rows of up to 8192): the next row is loaded before the sums
// over this one are joined, and the weights stay in registers (8,192 x 7168
// bf16: 119 us without either, 92 with the first, 85 with both; then near two
// thirds of the issue slots are busy).  1,024 threads leave 64 registers, of which
// fp32 rows, with twice the data in flight, spill 108 bytes and fp16 rows 20: 8,192 x
// 7168 take 232 us in fp32 (4.0 TB/s) and 102 in fp16.  Longer rows are read twice,
// the second time from L2: the registers hold dw.
template <typename T, int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) ep_norm_bwd_kernel(const NormParams p) {
  __shared__ float part[2][64];
  pdl_wait();
  const int vectors = p.H / 8, v0 = threadIdx.x;
  const T* weight = static_cast<const T*>(p.weight);
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  // Unsigned: the step past the last of 2^31 - 1 rows stays a number.
  const unsigned rows = static_cast<unsigned>(p.T);
  int turn = 0;
  if constexpr (NV == 1) {
    const bool in = v0 < vectors;
    float w[8];
    GradVec<T> next;
    if (in) {
      Raw8<T> wr;
      wr.load(weight + 8 * v0);
      wr.get(w);
      if (blockIdx.x < rows) next.load(p, blockIdx.x, v0, true);
    }
    for (unsigned t = blockIdx.x; t < rows; t += gridDim.x, turn ^= 1) {
      const GradVec<T> at = next;
      if (in && t + gridDim.x < rows) next.load(p, t + gridDim.x, v0, true);
      float ss = 0.0f, inner = 0.0f;
      if (in) at.sums(w, &ss, &inner);
      const float2 sums = block_sum2(ss, inner, part[turn]);
      const float r = 1.0f / sqrtf(sums.x / static_cast<float>(p.H) + p.eps);
      if (in) at.finish(p, t, v0, w, r, r * r * (sums.y / static_cast<float>(p.H)), dw[0]);
    }
  } else {
    for (unsigned t = blockIdx.x; t < rows; t += gridDim.x, turn ^= 1) {
      float ss = 0.0f, inner = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = v0 + i * blockDim.x;
        if (v < vectors) {
          GradVec<T> at;
          Raw8<T> wr;
          float w[8];
          at.load(p, t, v, false);
          wr.load(weight + 8 * v);
          wr.get(w);
          at.sums(w, &ss, &inner);
        }
      }
      const float2 sums = block_sum2(ss, inner, part[turn]);
      const float r = 1.0f / sqrtf(sums.x / static_cast<float>(p.H) + p.eps), c = r * r * (sums.y / static_cast<float>(p.H));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = v0 + i * blockDim.x;
        if (v < vectors) {
          GradVec<T> at;
          Raw8<T> wr;
          float w[8];
          at.load(p, t, v, true);
          wr.load(weight + 8 * v);
          wr.get(w);
          at.finish(p, t, v, w, r, c, dw[i]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + i * blockDim.x;
    if (v < vectors) store8<float>(p.partial + static_cast<long long>(blockIdx.x) * p.H + 8 * v, dw[i]);
  }
}

constexpr int kSumRows = 16;  // groups of partial rows per block, 32 columns wide

__global__ void __launch_bounds__(32 * kSumRows) ep_norm_dw_kernel(const NormParams p, int parts) {
  __shared__ float part[kSumRows][33];
  pdl_wait();
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float s = 0.0f;
  if (col < p.H) {
#pragma unroll 8
    for (int i = g; i < parts; i += kSumRows) s += p.partial[static_cast<long long>(i) * p.H + col];
  }
  part[g][threadIdx.x & 31] = s;
  __syncthreads();
  if (g == 0 && col < p.H) {
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) s += part[i][threadIdx.x];
    p.dw[col] = p.accumulate ? p.dw[col] + s : s;
  }
}

// Threads and vectors per thread for rows of H elements.  Two vectors a thread keep
// more loads of a batch in flight and its sum in fewer warps; one is quicker through
// the few rows of a decode step, fp32's vectors are twice as wide and do not care.
// bf16 with sum, y and q, 235 MB of x, and 128 rows: 2048 elements 167 us and 2.7
// (one vector: 183 and 2.2), 7168 168 and 3.2 (219 and 2.8), 1024 178 and 2.1 with
// the one that the rule takes (two: 166 and 2.7), 512 176 and 2.1 (181 and 2.5).  Four where 1,024
// threads need them: 16384 elements take 173 us with two, 201 with four.
void shape(int H, int* threads, int* nv) {
  const int vectors = H / 8;
  *nv = vectors <= 1024 ? 1 : vectors <= 2048 ? 2 : 4;
  if (vectors >= 256 && vectors <= 1024) *nv = 2;
  *threads = std::min(1024, ((vectors + *nv - 1) / *nv + 31) / 32 * 32);
}

template <typename T>
cudaError_t norm_typed(const NormParams& p, cudaStream_t s) {
  int threads, nv;
  shape(p.H, &threads, &nv);
  const dim3 grid(p.T), block(threads);
  if (nv == 1) return launch_pdl(ep_norm_kernel<T, 1>, grid, block, 0, s, 0, p);
  if (nv == 2) return launch_pdl(ep_norm_kernel<T, 2>, grid, block, 0, s, 0, p);
  return launch_pdl(ep_norm_kernel<T, 4>, grid, block, 0, s, 0, p);
}

template <typename T>
cudaError_t norm_bwd_typed(const NormParams& p, int parts, cudaStream_t s) {
  const int vectors = p.H / 8;
  const dim3 grid(parts);
  if (vectors <= 1024) return launch_pdl(ep_norm_bwd_kernel<T, 1>, grid, dim3((vectors + 31) / 32 * 32), 0, s, 0, p);
  if (vectors <= 2048) return launch_pdl(ep_norm_bwd_kernel<T, 4>, grid, dim3(512), 0, s, 0, p);
  return launch_pdl(ep_norm_bwd_kernel<T, 8>, grid, dim3(512), 0, s, 0, p);
}

// The expert of a receive row among offsets[0..E], by the warp: two rounds of
// 32 comparisons reach 1024 experts.
__device__ __forceinline__ int expert_of(const int* offsets, int E, int row, int lane) {
  const int step = (E + 31) / 32;
  const int above = __ballot_sync(kAll, lane * step < E && offsets[lane * step] <= row);
  const int base = (31 - __clz(above | 1)) * step;
  const unsigned in = __ballot_sync(kAll, lane < step && base + lane < E && offsets[base + lane] <= row);
  return base + 31 - __clz(in | 1);
}

// Eight lanes hold a block of 128, sixteen elements each.
__device__ __forceinline__ float quantize16(const float (&v)[2][8], uint4* q) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, max_nan(fabsf(v[0][i]), fabsf(v[1][i])));
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, d));
  const BlockScale s = block_scale(m);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* x = &v[i / 2][4 * (i & 1)];
    w[i] = e4m3x4(x[0] * s.inv, x[1] * s.inv, x[2] * s.inv, x[3] * s.inv);
  }
  *q = make_uint4(w[0], w[1], w[2], w[3]);
  return s.scale;
}

// A warp takes a row's segment of kSegment blocks of 128, four a step, sixteen
// elements a lane: with eight, stores of 8 bytes and twice the shuffles and
// quotients took 130 us for 32,768 receive rows of 7168 bf16 where these take 115
// (6.1 TB/s), and 79 for 65,536 of 2048 (70).  A row is loaded before it is known
// whether an expert owns it: 3% there, a microsecond lost where most are padding.
// Half or twice the segment, and one segment a warp without a stride, were slower.
constexpr int kQuantWarps = 8, kSegment = 8;

template <typename T>
__global__ void __launch_bounds__(kQuantWarps * 32) ep_quantize_kernel(const QuantParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int cols = scale_columns(p.n), segments = (cols + kSegment - 1) / kSegment;
  int rows = p.R;
  if (p.hdr != nullptr) {
    if (!blocks_ok(p.hdr, p.R)) return;
    rows = p.hdr[kHdrP];
  }
  const long long total = static_cast<long long>(rows) * segments;
  for (long long i = static_cast<long long>(blockIdx.x) * kQuantWarps + (threadIdx.x >> 5); i < total;
       i += static_cast<long long>(gridDim.x) * kQuantWarps) {
    const int row = static_cast<int>(i / segments), b0 = static_cast<int>(i - static_cast<long long>(row) * segments) * kSegment;
    const T* x = static_cast<const T*>(p.x) + static_cast<long long>(row) * p.n;
    Raw8<T> raw[kSegment / 4][2];
#pragma unroll
    for (int j = 0; j < kSegment / 4; ++j) {
      const int at = (b0 + 4 * j) * kF8Block + lane * 16;
      if (at < p.n) {
        raw[j][0].load(x + at);
        raw[j][1].load(x + at + 8);
      }
    }
    bool live = true;
    if (p.hdr != nullptr) {
      const int e = expert_of(p.offsets, p.E, row, lane);
      live = row - p.offsets[e] < p.counts[e];
    }
#pragma unroll
    for (int j = 0; j < kSegment / 4; ++j) {
      const int b = b0 + 4 * j + (lane >> 3), at = (b0 + 4 * j) * kF8Block + lane * 16;
      const bool in = live && at < p.n;
      float v[2][8] = {};
      if (in) {
        raw[j][0].get(v[0]);
        raw[j][1].get(v[1]);
      }
      uint4 q;
      const float s = quantize16(v, &q);
      if (at < p.n) *reinterpret_cast<uint4*>(p.q + static_cast<long long>(row) * p.n + at) = q;
      if ((lane & 7) == 0 && b < cols) p.scales[static_cast<long long>(row) * cols + b] = in ? s : 0.0f;
    }
  }
}

template <typename T>
cudaError_t quantize_typed(const QuantParams& p, int num_sms, cudaStream_t s) {
  const long long segments = (scale_columns(p.n) + kSegment - 1) / kSegment;
  const long long blocks = (p.R * segments + kQuantWarps - 1) / kQuantWarps;
  const unsigned grid = static_cast<unsigned>(std::min<long long>(blocks, 8LL * num_sms));
  return launch_pdl(ep_quantize_kernel<T>, dim3(grid), dim3(kQuantWarps * 32), 0, s, 0, p);
}

}  // namespace

// One to four blocks for each of 152 SMs, whatever the device has, so that the
// order of dw's sum does not depend on it: blocks of 513 to 1024 threads, 257 to
// 512 and fewer.
int norm_bwd_parts(long long T, long long H) {
  return static_cast<int>(std::min<long long>(T, H > 8192 ? 304 : H > 4096 ? 152 : H > 2048 ? 304 : 608));
}

cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP32) return norm_typed<float>(p, s);
  if (p.dtype == EP_DTYPE_FP16) return norm_typed<__half>(p, s);
  return norm_typed<__nv_bfloat16>(p, s);
}

cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s) {
  const int parts = norm_bwd_parts(p.T, p.H);
  if (parts > 0) {
    const cudaError_t e = p.dtype == EP_DTYPE_FP32   ? norm_bwd_typed<float>(p, parts, s)
                          : p.dtype == EP_DTYPE_FP16 ? norm_bwd_typed<__half>(p, parts, s)
                                                     : norm_bwd_typed<__nv_bfloat16>(p, parts, s);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(ep_norm_dw_kernel, dim3((p.H + 31) / 32), dim3(32 * kSumRows), 0, s, 0, p, parts);
}

cudaError_t launch_quantize(const QuantParams& p, int num_sms, cudaStream_t s) {
  if (p.dtype == EP_DTYPE_FP32) return quantize_typed<float>(p, num_sms, s);
  if (p.dtype == EP_DTYPE_FP16) return quantize_typed<__half>(p, num_sms, s);
  return quantize_typed<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace ep
