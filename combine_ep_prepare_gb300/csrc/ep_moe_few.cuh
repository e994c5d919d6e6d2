// ep_moe_few.cuh -- parameters and workspace of a few tokens' whole layer.
#pragma once

#include "ep_f8.cuh"

namespace ep {

constexpr int kFewBlocksMax = 256;  // of the second kernel
constexpr int kFewRows = 16;        // weight rows of one piece of its work

struct FewParams {
  int T, E, K, H, F, dtype, gate_dtype, f8;
  RouterParams router;   // logits are the workspace's
  const void* x;
  const void* gate;
  const void* w13;
  const float* s13;
  const void* w2;
  const float* s2;
  void* out;
  long long* idx;
  float* w;
  // workspace
  int* hdr;              // [0] status, [1] arrivals of the second kernel's blocks
  int* done;             // [tiles of 16 outputs] blocks that have added their part
  int* written;          // 8-bit weights: [used expert][blocks of F] pieces of act there, where blocks share them
  int zeros;             // ints from hdr on that the first kernel zeroes
  float* logits;         // [T][E]
  void* act;             // [routes][F], an expert's routes side by side: payload, or float32 with 8-bit weights
  __half* xq;            // 8-bit weights: [T][H], e4m3 values in fp16
  float* xs;             // [T][scale_columns(H)]
  __half* aq;            // [routes][F], the same
  float* as;             // [routes][scale_columns(F)]
  float* part;           // [blocks][2][16][T]: sums of the outputs that several blocks share
};

struct FewLayout {
  size_t done, written, logits, act, xq, xs, aq, as, part, total;
  int zeros;
};
inline FewLayout few_layout(long long T, long long E, long long K, long long H, long long F, bool f8) {
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const long long routes = T * K, used = E < routes ? E : routes;
  FewLayout l;
  size_t at = 256;
  l.done = at;
  at += static_cast<size_t>((H + kFewRows - 1) / kFewRows) * 4;
  l.written = at;
  if (f8) at += static_cast<size_t>(used * f8_blocks(static_cast<int>(F))) * 4;
  l.zeros = static_cast<int>(at / 4);
  at = up(at);
  l.logits = at;
  at = up(at + T * E * 4);
  l.act = at;
  at = up(at + routes * F * 4);
  l.part = at;
  at = up(at + static_cast<size_t>(kFewBlocksMax) * 2 * kFewRows * T * 4);
  l.xq = at;
  if (f8) at = up(at + T * H * 2);
  l.xs = at;
  if (f8) at = up(at + T * scale_columns(static_cast<int>(H)) * 4);
  l.aq = at;
  if (f8) at = up(at + routes * F * 2);
  l.as = at;
  if (f8) at = up(at + routes * scale_columns(static_cast<int>(F)) * 4);
  l.total = at;
  return l;
}

cudaError_t launch_moe_few(const FewParams& p, int num_sms, cudaStream_t s);

}  // namespace ep
