// Argument checks and small device helpers shared by the plan-less operators (rotary append,
// tree attention, cache pages).
#pragma once

#include <atomic>

#include "launch.h"

namespace gqa {

inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Is `device` one the call can run on?
inline gqa_status_t check_device(int device) {
  static std::atomic<int> known{0};  // devices the process sees; it does not change
  int ndev = known.load(std::memory_order_relaxed);
  if (ndev == 0) {
    if (cudaGetDeviceCount(&ndev) != cudaSuccess) {
      cudaGetLastError();
      return GQA_ERR_CUDA;
    }
    known.store(ndev, std::memory_order_relaxed);
  }
  if (device < 0 || device >= ndev) return GQA_ERR_INVALID_ARG;
  return GQA_OK;
}

// The geometry checks of a [B, T, H, 128] call over a cache (as gqa_prefill_attn's).
inline gqa_status_t check_cache_geometry(int batch, int num_q_heads, int num_kv_heads, int head_dim, int tokens,
                                         int block_size, int max_seq_len, int num_cache_blocks) {
  if (head_dim != kHeadDim) return GQA_ERR_UNSUPPORTED;
  if (batch < 1 || batch > GQA_MAX_BATCH || num_q_heads < 1 || num_kv_heads < 1 || tokens < 1 || max_seq_len < 1 ||
      tokens > max_seq_len)
    return GQA_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > GQA_MAX_GROUP) return GQA_ERR_UNSUPPORTED;
  if (block_size != 0 && block_size != GQA_BLOCK_SIZE) return GQA_ERR_UNSUPPORTED;
  if (block_size > 0 && num_cache_blocks < 1) return GQA_ERR_INVALID_ARG;
  const long long rows = block_size > 0 ? static_cast<long long>(num_cache_blocks) * kTile
                                        : static_cast<long long>(batch) * max_seq_len;
  if (rows > 0x7fffffffLL || static_cast<long long>(batch) * tokens > 0x7fffffffLL) return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

// Sets bits in the caller's error word, if it gave one.
__device__ __forceinline__ void flag_error(uint32_t *err, uint32_t bits) {
  if (err) atomicOr(err, bits);
}

}  // namespace gqa
