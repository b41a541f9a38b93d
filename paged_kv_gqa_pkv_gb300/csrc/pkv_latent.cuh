// pkv_latent.cuh - what the operators of a paged cache of shared latents have in
// common: the row's sizes, the cache's checks, and waits with a limit.
//
// A cache row is one token's latent (kLatent values, key and value of every head)
// and its rotated position part (kRotated values, key only), bf16.
#pragma once

#include <climits>

#include "pkv_prefill_common.cuh"

namespace pkv {
namespace latent {

constexpr int kLatent = 512;
constexpr int kRotated = 64;
constexpr int kRow = kLatent + kRotated;  // 576 values, 1152 bytes
constexpr int kOwnKey = 128;              // expanded: a head's own part of a key
constexpr int kValue = 128;               // expanded: a head's value

// PKV_OK for a geometry that the latent calls serve.
inline pkv_status check_latent_cache(const pkv_cache_desc* c) {
  if (c == nullptr) return PKV_ERR_ARG;
  if (c->num_pages <= 0 || c->page_size <= 0 || c->page_size % 16 != 0) return PKV_ERR_ARG;
  if (c->num_kv_heads != 1 || c->head_dim != kRow) return PKV_ERR_ARG;
  if (c->max_batch <= 0 || c->max_blocks <= 0) return PKV_ERR_ARG;
  if (static_cast<long long>(c->num_pages) * c->page_size > INT_MAX) return PKV_ERR_ARG;
  if (static_cast<long long>(c->max_blocks) * c->page_size > INT_MAX) return PKV_ERR_ARG;
  if (static_cast<long long>(c->max_batch) * c->max_blocks > INT_MAX) return PKV_ERR_ARG;
  return PKV_OK;
}

inline bool is_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// The limit of a wait. Reading the global timer takes hundreds of cycles, so it is read only
// every 256th time that there is nothing to do.
struct WaitLimit {
  uint64_t since = 0;
  uint32_t n = 0;
  __device__ __forceinline__ bool over(volatile int* abort_flag) {
    if ((++n & 255u) != 0) return false;
    const uint64_t now = global_timer_ns();
    if (since == 0) since = now;
    if (*abort_flag == 0 && now - since <= kWaitLimitNs) return false;
    *abort_flag = 1;
    return true;
  }
};

// Waits for a phase; false once the limit is over or another role of the CTA has given up.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity,
                                           volatile int* abort_flag) {
  WaitLimit limit;
  while (!mbar_try_wait(bar, parity))
    if (limit.over(abort_flag)) return false;
  return true;
}

}  // namespace latent
}  // namespace pkv
