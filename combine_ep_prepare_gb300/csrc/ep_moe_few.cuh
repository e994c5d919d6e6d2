// ep_moe_few.cuh -- parameters and workspace of a few tokens' whole layer.
#pragma once

#include "ep_f8.cuh"

namespace ep {

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
  float* logits;         // [T][E]
  float* act;            // [routes][F], an expert's routes side by side
  uint8_t* xq;           // 8-bit weights: [T][H]
  float* xs;             // [T][scale_columns(H)]
};

struct FewLayout {
  size_t logits, act, xq, xs, total;
};
inline FewLayout few_layout(long long T, long long E, long long K, long long H, long long F, bool f8) {
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  FewLayout l;
  size_t at = 256;
  l.logits = at;
  at = up(at + T * E * 4);
  l.act = at;
  at = up(at + T * K * F * 4);
  l.xq = at;
  if (f8) at = up(at + T * H);
  l.xs = at;
  if (f8) at = up(at + T * scale_columns(static_cast<int>(H)) * 4);
  l.total = at;
  return l;
}

cudaError_t launch_moe_few(const FewParams& p, int num_sms, cudaStream_t s);

}  // namespace ep
