// ep_api_checks.h -- argument checks shared by the C ABI's translation units
// outside ep_api.cu.
#pragma once

#include <cstdio>

#include "ep_experts.cuh"

namespace ep {
namespace checks {

inline bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

inline ep_status_t fail(ep_status_t code, const char* fmt, const char* name, long long v = 0) {
  char buf[256];
  snprintf(buf, sizeof buf, fmt, name, v);
  return api_fail(code, buf);
}

inline ep_status_t check_ptr(const void* p, const char* name, size_t align = 16) {
  if (p == nullptr) return fail(EP_ERR_INVALID_ARG, "%s is NULL", name);
  if (misaligned(p, align)) return fail(EP_ERR_INVALID_ARG, "%s is not %lld-byte aligned", name, (long long)align);
  return EP_OK;
}

template <typename T>
T* at(void* mem, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(mem) + off); }

inline int own_experts(const LayerInfo* L) {
  return static_cast<int>(L->nranks > 0 ? L->cfg.num_experts / L->nranks : L->cfg.num_experts);
}

// A router's configuration and tokens; logits are checked by the caller.
ep_status_t router_config(const ep_router_config_t& c, int64_t T, RouterParams* p);

}  // namespace checks
}  // namespace ep
