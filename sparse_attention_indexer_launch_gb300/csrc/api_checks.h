// Argument checks that the verify step's entry points share (tree_api.cu, step_api.cu).
#pragma once

#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "idx.h"

namespace idx {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool words(std::initializer_list<const void *> arrays) {   // 4-byte elements at 4-byte addresses (or null)
  for (const void *p : arrays)
    if (!aligned(p, 4)) return false;
  return true;
}

inline idx_status cuda_ok(cudaError_t e) { return e == cudaSuccess ? IDX_OK : IDX_ECUDA; }

constexpr size_t kStateAlign = 1024;
constexpr size_t kStatusBytes = 1024;   // the status word's block at the start of every state

inline bool state_ok(const void *state, size_t bytes, size_t need) {
  return state != nullptr && aligned(state, kStateAlign) && bytes >= need;
}

// keys_alone: a cache without values is taken too.
inline idx_status check_cache(const idx_kv_cache *c, bool keys_alone = false) {
  const bool has_v = c->v != nullptr || !keys_alone;
  if (c->k == nullptr || !aligned(c->k, 16)) return IDX_EINVAL;
  if (has_v && (c->v == nullptr || !aligned(c->v, 16))) return IDX_EINVAL;
  if (c->P < 1 || c->Hkv < 1) return IDX_EINVAL;
  if (c->P > INT32_MAX / IDX_PAGE || c->Hkv > 1024) return IDX_EUNSUPPORTED;
  if (c->D != 64 && c->D != 128) return IDX_EUNSUPPORTED;
  int64_t bytes;
  if (c->kv_dtype == IDX_KV_E4M3) {
    bytes = 1;
    if (c->k_scale == nullptr || !aligned(c->k_scale, 16)) return IDX_EINVAL;
    if (has_v ? c->v_scale == nullptr || !aligned(c->v_scale, 16) : c->v_scale != nullptr) return IDX_EINVAL;
  } else if (c->kv_dtype == IDX_KV_BF16) {
    bytes = 2;
    if (c->k_scale != nullptr || c->v_scale != nullptr) return IDX_EINVAL;
  } else {
    return IDX_EINVAL;
  }
  for (const int64_t s : {c->page_stride, c->token_stride, c->head_stride}) {
    if (s < 1 || s % (16 / bytes) != 0) return IDX_EINVAL;
    if (s >= (int64_t{1} << 40) / bytes) return IDX_EUNSUPPORTED;   // a tensor map's strides have 40 bits
  }
  return IDX_OK;
}

}  // namespace idx
