// The C ABI of the verify step's two ends (include/idx.h): argument checks and launches.
#include <cmath>

#include "api_checks.h"
#include "idx.h"
#include "idx_device.cuh"
#include "launch.h"

namespace {

using idx::aligned;
using idx::check_cache;
using idx::cuda_ok;
using idx::kStatusBytes;
using idx::state_ok;
using idx::words;

// One of q, k, v or an output: rows of `heads` heads.
bool rows_ok(const void *p, int64_t stride, int64_t heads, int64_t D) {
  return p != nullptr && aligned(p, 16) && stride >= heads * D && stride % 8 == 0;
}
constexpr int64_t kMaxStride = int64_t{1} << 39;   // elements: a row's offset stays within 64 bits

idx_status check_norm_rope(const idx_norm_rope_args *p, const idx_kv_cache *c) {
  if (p == nullptr || p->R < 0) return IDX_EINVAL;
  if (c != nullptr) {
    const idx_status st = check_cache(c, true);
    if (st != IDX_OK) return st;
    if (c->Hkv != p->Hkv || c->D != p->D) return IDX_EINVAL;
  }
  const bool has_v = c != nullptr && c->v != nullptr;
  if (p->Hq < 0 || p->Hkv < 0 || p->Hq + static_cast<int64_t>(p->Hkv) < 1) return IDX_EINVAL;
  if (p->Hq > 1024 || p->Hkv > 1024) return IDX_EUNSUPPORTED;
  if (p->D != 64 && p->D != 128 && p->D != 256) return IDX_EUNSUPPORTED;
  if (p->rot < 0 || p->rot > p->D) return IDX_EINVAL;
  if (p->rot % 16 != 0) return IDX_EUNSUPPORTED;   // pairs of whole lanes
  if (p->axes < 1 || p->axes > IDX_MAX_AXES) return IDX_EINVAL;
  for (int i = 0; i < p->rot / 2; ++i)
    if (p->axis[i] >= p->axes) return IDX_EINVAL;
  for (const int n : {p->q_norm, p->k_norm})
    if (n != IDX_NORM_NONE && n != IDX_NORM_RMS && n != IDX_NORM_LAYER) return IDX_EINVAL;
  if ((p->q_weight != nullptr && p->q_norm == IDX_NORM_NONE) || (p->k_weight != nullptr && p->k_norm == IDX_NORM_NONE) ||
      (p->q_bias != nullptr && p->q_norm != IDX_NORM_LAYER) || (p->k_bias != nullptr && p->k_norm != IDX_NORM_LAYER))
    return IDX_EINVAL;
  if (!(p->eps >= 0x1p-60f && p->eps <= 1.0f)) return IDX_EINVAL;
  if (p->R == 0) return IDX_OK;
  for (const float *w : {p->q_weight, p->q_bias, p->k_weight, p->k_bias})
    if (!aligned(w, 16)) return IDX_EINVAL;
  if (!words({p->pos, p->inv_freq, p->slot, p->rows})) return IDX_EINVAL;
  if (p->Hq > 0) {
    if (!rows_ok(p->q, p->q_stride, p->Hq, p->D) || !rows_ok(p->q_out, p->q_out_stride, p->Hq, p->D)) return IDX_EINVAL;
    if (p->q == p->q_out && p->q_stride != p->q_out_stride) return IDX_EINVAL;
  } else if (p->q != nullptr || p->q_out != nullptr) {
    return IDX_EINVAL;
  }
  if (p->Hkv > 0) {
    if (!rows_ok(p->k, p->k_stride, p->Hkv, p->D)) return IDX_EINVAL;
    if (p->k_out != nullptr && !rows_ok(p->k_out, p->k_out_stride, p->Hkv, p->D)) return IDX_EINVAL;
    if (p->k == p->k_out && p->k_stride != p->k_out_stride) return IDX_EINVAL;
    if (p->k_out == nullptr && c == nullptr) return IDX_EINVAL;   // keys that go nowhere
  } else if (p->k != nullptr || p->k_out != nullptr) {
    return IDX_EINVAL;
  }
  if (has_v ? !rows_ok(p->v, p->v_stride, p->Hkv, p->D) : p->v != nullptr) return IDX_EINVAL;
  if ((c != nullptr) != (p->slot != nullptr)) return IDX_EINVAL;
  if (p->rot > 0 && (p->pos == nullptr || p->inv_freq == nullptr)) return IDX_EINVAL;
  if (p->pos_stride < 0 || (p->axes > 1 && p->pos_stride < p->R)) return IDX_EINVAL;
  // a warp per vector at most: their number stays below 2^31
  if (p->R > INT32_MAX / (p->Hq + 2 * static_cast<int64_t>(p->Hkv))) return IDX_EUNSUPPORTED;
  for (const int64_t s : {p->q_stride, p->k_stride, p->v_stride, p->q_out_stride, p->k_out_stride, p->pos_stride})
    if (s >= kMaxStride) return IDX_EUNSUPPORTED;
  return IDX_OK;
}

idx_status check_sample(const idx_sample_args *p, const int32_t *token, const float *logprob) {
  if (p == nullptr || p->logits == nullptr || p->u == nullptr || token == nullptr) return IDX_EINVAL;
  if (p->logits_dtype != IDX_LOGITS_F32 && p->logits_dtype != IDX_LOGITS_BF16) return IDX_EINVAL;
  if (p->R < 1 || p->V < 1 || p->ld < p->V) return IDX_EINVAL;
  if (!aligned(p->logits, p->logits_dtype == IDX_LOGITS_F32 ? 4 : 2)) return IDX_EINVAL;
  if (!words({p->u, p->temperature, p->top_p, p->min_p, p->top_k, p->rows, token, logprob})) return IDX_EINVAL;
  if (p->R > IDX_MAX_ROWS || p->V > IDX_MAX_VOCAB || p->ld >= kMaxStride) return IDX_EUNSUPPORTED;
  return IDX_OK;
}

}  // namespace

extern "C" {

idx_status idx_norm_rope(const idx_norm_rope_args *args, const idx_kv_cache *cache, void *stream) {
  idx_status st = check_norm_rope(args, cache);
  if (st != IDX_OK || args->R == 0) return st;
  int sms = 0;
  st = idx::device_sms(&sms);
  if (st != IDX_OK) return st;
  idx::NormRopeArgs a{};
  a.p = *args;
  if (cache != nullptr) a.c = *cache;
  return cuda_ok(idx::launch_norm_rope(a, sms, static_cast<cudaStream_t>(stream)));
}

idx_status idx_sample(const idx_sample_args *args, int32_t *token, float *logprob, void *stream) {
  idx_status st = check_sample(args, token, logprob);
  if (st != IDX_OK) return st;
  int sms = 0;
  st = idx::device_sms(&sms);   // the device check
  if (st != IDX_OK) return st;
  idx::SampleArgs a{};
  a.p = *args;
  a.token = token;
  a.logprob = logprob;
  a.vec = args->ld % 4 == 0 && aligned(args->logits, args->logits_dtype == IDX_LOGITS_F32 ? 16 : 8);
  return cuda_ok(idx::launch_sample(a, static_cast<cudaStream_t>(stream)));
}

size_t idx_tree_accept_state_size(void) { return kStatusBytes; }

idx_status idx_tree_accept(const idx_tree_accept_args *t, void *state, size_t state_bytes, void *stream) {
  if (t == nullptr || t->row_start == nullptr || t->draft == nullptr || t->target == nullptr || t->ctx_len == nullptr ||
      t->page_table == nullptr || t->free_pages == nullptr || t->free_count == nullptr || t->new_ctx == nullptr ||
      t->free_left == nullptr || t->accept_len == nullptr || t->last == nullptr || t->path == nullptr || t->token == nullptr)
    return IDX_EINVAL;
  if (!words({t->row_start, t->parent, t->draft, t->target, t->ctx_len, t->page_table, t->free_pages, t->free_count, t->new_ctx,
              t->free_left, t->accept_len, t->last, t->path, t->token}))
    return IDX_EINVAL;
  if (t->Q < 1 || t->P < 1 || t->pt_stride < 1 || t->cap < 1 || t->free_cap < 0) return IDX_EINVAL;
  // the walk of one request reads what another's would overwrite
  if (t->path == t->draft || t->path == t->target || t->token == t->draft || t->token == t->target || t->path == t->token)
    return IDX_EINVAL;
  if (t->Q > IDX_MAX_REQS || t->P > INT32_MAX / IDX_PAGE || t->cap > INT32_MAX - 3) return IDX_EUNSUPPORTED;
  if (!state_ok(state, state_bytes, kStatusBytes)) return IDX_EINVAL;
  int sms = 0;
  const idx_status st = idx::device_sms(&sms);
  if (st != IDX_OK) return st;
  idx::TreeAcceptArgs a{};
  a.t = *t;
  a.status = static_cast<uint32_t *>(state);
  a.arrived = a.status + 1;
  return cuda_ok(idx::launch_tree_accept(a, sms, static_cast<cudaStream_t>(stream)));
}

idx_status idx_tree_commit(const idx_kv_cache *cache, const int32_t *row_start, const int32_t *accept_len, const int32_t *path,
                           const int32_t *slot, int32_t Q, int32_t cap, void *stream) {
  if (cache == nullptr || row_start == nullptr || accept_len == nullptr || path == nullptr || slot == nullptr) return IDX_EINVAL;
  idx_status st = check_cache(cache, true);
  if (st != IDX_OK) return st;
  if (!words({row_start, accept_len, path, slot}) || Q < 1 || cap < 1) return IDX_EINVAL;
  if (Q > IDX_MAX_REQS || cap > INT32_MAX - 3) return IDX_EUNSUPPORTED;
  int sms = 0;
  st = idx::device_sms(&sms);   // the device check
  if (st != IDX_OK) return st;
  idx::TreeCommitArgs a{};
  a.c = *cache;
  a.row_start = row_start;
  a.accept_len = accept_len;
  a.path = path;
  a.slot = slot;
  a.Q = Q;
  a.cap = cap;
  return cuda_ok(idx::launch_tree_commit(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
