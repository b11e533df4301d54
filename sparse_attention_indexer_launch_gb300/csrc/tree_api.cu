// The C ABI of the tree-verify step (include/idx.h): argument checks and launches.
#include <cuda.h>

#include <cmath>
#include <initializer_list>

#include "idx.h"
#include "idx_device.cuh"
#include "launch.h"

namespace {

constexpr size_t kStateAlign = 1024;
constexpr int kMaxGroup = 128;          // query heads per key/value head: the rows of a tensor-core tile
constexpr size_t kStatusBytes = 1024;   // the status word's block at the start of every state
constexpr int32_t kMaxCtx = 1 << 30;    // cached tokens of a request: its keys, up to the end of a tile, fit 31 bits

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool words(std::initializer_list<const void *> arrays) {   // 4-byte elements at 4-byte addresses (or null)
  for (const void *p : arrays)
    if (!aligned(p, 4)) return false;
  return true;
}

idx_status cuda_ok(cudaError_t e) { return e == cudaSuccess ? IDX_OK : IDX_ECUDA; }

bool state_ok(const void *state, size_t bytes, size_t need) {
  return state != nullptr && aligned(state, kStateAlign) && bytes >= need;
}

idx_status check_cache(const idx_kv_cache *c) {
  if (c->k == nullptr || c->v == nullptr || !aligned(c->k, 16) || !aligned(c->v, 16)) return IDX_EINVAL;
  if (c->P < 1 || c->Hkv < 1) return IDX_EINVAL;
  if (c->P > INT32_MAX / IDX_PAGE || c->Hkv > 1024) return IDX_EUNSUPPORTED;
  if (c->D != 64 && c->D != 128) return IDX_EUNSUPPORTED;
  int64_t bytes;
  if (c->kv_dtype == IDX_KV_E4M3) {
    bytes = 1;
    if (c->k_scale == nullptr || c->v_scale == nullptr || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
      return IDX_EINVAL;
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

// The launch's shape.  Up to 64 rows of a request and key/value head (selected: of a token)
// go to the few-row kernel, over a bf16 cache up to 32; up to 128 rows to the many-row kernel in
// one block, more in pairs of blocks that share every K and V tile (4 requests of 64 x 64 rows:
// 184 us, one block at a time 206; E4M3, 2 x 64 x 64 rows on 2 heads: 225, 294).  Few-row
// against many-row kernel, us, 4 tokens, 8 key/value heads:
//                          1 request, 131,072 keys   32 requests, 1,024 to 16,384 keys
//   bf16 D =  64, 32 rows         62    76                   99   116
//   bf16 D = 128, 32 rows         96    99                  156   154
//   bf16 D =  64, 64 rows         71    80                  143   121
//   bf16 D = 128, 64 rows        107   100                  205   164
//   E4M3 D =  64, 32 rows         73   136                  127   238
//   E4M3 D = 128, 32 rows         85   154                  167   282
//   E4M3 D =  64, 64 rows        111   138                  220   259
//   E4M3 D = 128, 64 rows        130   160                  274   317
// One long request of 64 rows at D = 64 would be served faster by the few-row kernel, batches
// lose more there.
struct Shape {
  int rows;           // the few-row kernel's N, or 0
  int tile;           // keys
  int block_tokens;   // tokens of a row block
  bool pair;
};
Shape shape_of(const idx_tree_problem *p, int32_t sel_k) {
  Shape s{};
  const int G = p->Hq / p->cache.Hkv;
  const int rows = (sel_k > 0 ? 1 : p->max_new) * G;
  if (rows <= (sel_k > 0 || p->cache.kv_dtype == IDX_KV_E4M3 ? 64 : 32)) {
    s.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    s.tile = 128;
    s.block_tokens = sel_k > 0 ? 1 : s.rows / G;
  } else {
    s.tile = IDX_PAGE;
    s.block_tokens = sel_k > 0 ? 1 : kMaxGroup / G;
    s.pair = rows > s.block_tokens * G;
  }
  return s;
}

// Tiles of the launch, at most: the kernels count them in 31 bits, and take INT32_MAX for more.
bool tiles_fit(const idx_tree_problem *p, int32_t sel_k) {
  const Shape s = shape_of(p, sel_k);
  const int64_t item = s.pair ? 2 * s.block_tokens : s.block_tokens;
  const int64_t tiles = ((sel_k > 0 ? sel_k : p->max_ctx) + static_cast<int64_t>(p->max_new) + s.tile - 1) / s.tile;
  const int64_t blocks = (p->max_new + item - 1) / item;
  const int64_t items = (static_cast<int64_t>(p->Q) * blocks < p->R ? static_cast<int64_t>(p->Q) * blocks : p->R) * p->cache.Hkv;
  return items * tiles < INT32_MAX;
}

idx_status check_problem(const idx_tree_problem *p, int32_t sel_k) {
  if (p == nullptr) return IDX_EINVAL;
  if (p->q == nullptr || !aligned(p->q, 16) || p->page_table == nullptr || p->ctx_len == nullptr ||
      p->row_start == nullptr)
    return IDX_EINVAL;
  if (!words({p->page_table, p->ctx_len, p->row_start}) || !aligned(p->mask, 8)) return IDX_EINVAL;
  const idx_status st = check_cache(&p->cache);
  if (st != IDX_OK) return st;
  if (p->R < 1 || p->Q < 1 || p->pt_stride < 1 || p->max_ctx < 0 || p->max_new < 1 || p->Hq < 1) return IDX_EINVAL;
  if (static_cast<int64_t>(p->max_ctx) > static_cast<int64_t>(p->pt_stride) * IDX_PAGE) return IDX_EINVAL;
  if (p->Hq % p->cache.Hkv != 0 || !std::isfinite(p->scale) || p->scale < 0.0f) return IDX_EINVAL;
  if (p->q_row_stride < static_cast<int64_t>(p->Hq) * p->cache.D || p->q_row_stride % 8 != 0) return IDX_EINVAL;
  if (p->R > IDX_MAX_ROWS || p->Q > IDX_MAX_REQS || p->max_new > IDX_MAX_TREE || p->Hq > 1024) return IDX_EUNSUPPORTED;
  if (sel_k < 0 || sel_k > IDX_MAX_K) return IDX_EINVAL;
  if (p->max_ctx > kMaxCtx) return IDX_EUNSUPPORTED;
  if (p->Hq / p->cache.Hkv > kMaxGroup) return IDX_EUNSUPPORTED;
  if (!tiles_fit(p, sel_k)) return IDX_EUNSUPPORTED;
  if (p->q_row_stride >= int64_t{1} << 39) return IDX_EUNSUPPORTED;   // a tensor map's strides have 40 bits
  return IDX_OK;
}

size_t round_up(size_t x) { return (x + kStateAlign - 1) / kStateAlign * kStateAlign; }

struct StateLayout {
  size_t joins, ml, o, total;
};
StateLayout state_layout(const idx_tree_problem *p, int32_t sel_k) {
  const Shape s = shape_of(p, sel_k);
  const size_t slots = 2 * static_cast<size_t>(idx::kTreeMaxCtas) * (s.pair ? 256 : 128);
  StateLayout L{};
  L.joins = kStatusBytes;
  L.ml = L.joins + round_up(idx::kTreeMaxCtas * sizeof(uint2));
  L.o = L.ml + round_up(slots * sizeof(float2));
  L.total = L.o + round_up(slots * p->cache.D * sizeof(float));
  return L;
}

// What the tensor core reads is swizzled by rows of 128 bytes (bf16: boxes of 64 dimensions;
// E4M3 K of 128 dimensions) or 64 bytes (E4M3 K of 64 dimensions); E4M3 V is converted in
// shared memory and comes as it is.
CUtensorMapSwizzle cache_swizzle(const idx_kv_cache *c, bool is_v) {
  if (c->kv_dtype == IDX_KV_BF16) return CU_TENSOR_MAP_SWIZZLE_128B;
  if (is_v) return CU_TENSOR_MAP_SWIZZLE_NONE;
  return c->D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
}

// K or V as a 4-D tensor [P][Hkv][64][D].  L2 fetches no more around a head's row than the
// row, unless its tokens lie next to each other.
idx_status cache_map(PFN_cuTensorMapEncodeTiled_v12000 encode, const idx_kv_cache *c, bool is_v, CUtensorMap *map) {
  void *const base = is_v ? c->v : c->k;
  const bool f8 = c->kv_dtype == IDX_KV_E4M3;
  const cuuint64_t e = f8 ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->D), IDX_PAGE, static_cast<cuuint64_t>(c->Hkv),
                              static_cast<cuuint64_t>(c->P)};
  const cuuint64_t strides[3] = {c->token_stride * e, c->head_stride * e, c->page_stride * e};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(f8 ? c->D : 64), IDX_PAGE, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const cuuint64_t run = c->token_stride == c->D ? 256 : c->D * e;   // bytes of a head next to each other
  const CUtensorMapL2promotion promote = run >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                         : run >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                      : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  const CUresult r = encode(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
                            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            cache_swizzle(c, is_v), promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? IDX_OK : IDX_ECUDA;
}

idx_status attend(const idx_tree_problem *p, const int32_t *sel, int32_t sel_k, void *out, float *lse, void *state,
                  size_t state_bytes, void *stream) {
  idx_status st = check_problem(p, sel_k);
  if (st != IDX_OK) return st;
  const StateLayout L = state_layout(p, sel_k);
  if (out == nullptr || !aligned(out, 16) || !words({sel, lse}) || !state_ok(state, state_bytes, L.total)) return IDX_EINVAL;
  int sms = 0;
  st = idx::device_sms(&sms);
  if (st != IDX_OK) return st;
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  st = idx::tensor_map_encoder(&encode);
  if (st != IDX_OK) return st;
  const Shape s = shape_of(p, sel_k);
  const int D = p->cache.D, G = p->Hq / p->cache.Hkv;
  CUtensorMap qm{}, km{}, vm{};
  if (p->cache.kv_dtype == IDX_KV_BF16) {   // beside an E4M3 cache Q is split as it is loaded
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p->Hq), static_cast<cuuint64_t>(p->R)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(p->q_row_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(s.block_tokens)};
    const cuuint32_t one[3] = {1, 1, 1};
    if (encode(&qm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p->q), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return IDX_ECUDA;
  }
  uint8_t *const b = static_cast<uint8_t *>(state);
  idx::TreeAttnArgs a{};
  if (sel == nullptr) {
    st = cache_map(encode, &p->cache, false, &km);
    if (st == IDX_OK) st = cache_map(encode, &p->cache, true, &vm);
  }   // selected positions are gathered by plain loads
  if (st != IDX_OK) return st;
  a.p = *p;
  a.sel = sel;
  a.sel_k = sel_k;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.status = static_cast<uint32_t *>(state);
  a.joins = reinterpret_cast<uint2 *>(b + L.joins);
  a.part_ml = reinterpret_cast<float2 *>(b + L.ml);
  a.part_o = reinterpret_cast<float *>(b + L.o);
  a.wait_limit_ns = idx::device_wait_limit_ns();
  a.pair = s.pair;
  a.tile = s.tile;
  a.rows = s.rows;
  a.item_tokens = s.pair ? 2 * s.block_tokens : s.block_tokens;
  const int ctas = sms < idx::kTreeMaxCtas ? sms : idx::kTreeMaxCtas;
  const bool f8 = p->cache.kv_dtype == IDX_KV_E4M3;
  idx::TreeAttnLaunch *const launches[2][2][2] = {   // [many][E4M3][D = 128]
      {{idx::launch_tree_few_bf16_64, idx::launch_tree_few_bf16_128}, {idx::launch_tree_few_e4m3_64, idx::launch_tree_few_e4m3_128}},
      {{idx::launch_tree_many_bf16_64, idx::launch_tree_many_bf16_128},
       {idx::launch_tree_many_e4m3_64, idx::launch_tree_many_e4m3_128}}};
  idx::TreeAttnLaunch *const launch = launches[s.rows == 0][f8][D == 128];
  return cuda_ok(launch(a, qm, km, vm, ctas, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t idx_tree_tables_state_size(void) { return kStatusBytes; }

idx_status idx_tree_tables(const idx_tree_tables_args *t, void *state, size_t state_bytes, void *stream) {
  if (t == nullptr || t->ctx_len == nullptr || t->new_len == nullptr || t->free_pages == nullptr ||
      t->free_count == nullptr || t->page_table == nullptr || t->row_start == nullptr || t->free_left == nullptr)
    return IDX_EINVAL;
  if (t->Q < 1 || t->P < 1 || t->pt_stride < 1 || t->cap < 0) return IDX_EINVAL;
  if (t->cap > 0 && (t->row_req == nullptr || t->row_bound == nullptr || t->row_pos == nullptr || t->slot == nullptr))
    return IDX_EINVAL;
  if (t->free_left == t->free_count || !aligned(t->mask, 8)) return IDX_EINVAL;
  if (!words({t->ctx_len, t->new_len, t->parent, t->free_pages, t->free_count, t->page_table, t->row_start, t->free_left,
              t->row_req, t->row_bound, t->row_pos, t->slot}))
    return IDX_EINVAL;
  if (t->Q > IDX_MAX_REQS || t->P > INT32_MAX / IDX_PAGE) return IDX_EUNSUPPORTED;
  if (t->cap > INT32_MAX - 3) return IDX_EUNSUPPORTED;   // a thread's four rows end within 31 bits
  if (!state_ok(state, state_bytes, kStatusBytes)) return IDX_EINVAL;
  int sms = 0;
  const idx_status st = idx::device_sms(&sms);
  if (st != IDX_OK) return st;
  idx::TreeTablesArgs a{};
  a.t = *t;
  a.status = static_cast<uint32_t *>(state);
  a.vec4 = aligned(t->row_req, 16) && aligned(t->row_bound, 16) && aligned(t->row_pos, 16) && aligned(t->slot, 16) &&
           aligned(t->mask, 16);
  return cuda_ok(idx::launch_tree_tables(a, sms, static_cast<cudaStream_t>(stream)));
}

idx_status idx_write_kv(const idx_kv_cache *cache, const void *k_new, const void *v_new, int64_t row_stride,
                        const int32_t *slot, int64_t R, void *stream) {
  if (cache == nullptr || R < 0) return IDX_EINVAL;
  idx_status st = check_cache(cache);
  if (st != IDX_OK) return st;
  if (R == 0) return IDX_OK;
  if (k_new == nullptr || v_new == nullptr || slot == nullptr || !aligned(k_new, 16) || !aligned(v_new, 16) || !words({slot}))
    return IDX_EINVAL;
  if (row_stride < static_cast<int64_t>(cache->Hkv) * cache->D || row_stride % 8 != 0) return IDX_EINVAL;
  if (R > INT32_MAX) return IDX_EUNSUPPORTED;   // the grid: a row is at most 128 CTAs of vectors
  int sms = 0;
  st = idx::device_sms(&sms);   // the device check
  if (st != IDX_OK) return st;
  idx::WriteKvArgs a{};
  a.c = *cache;
  a.k_new = static_cast<const uint16_t *>(k_new);
  a.v_new = static_cast<const uint16_t *>(v_new);
  a.row_stride = row_stride;
  a.R = R;
  a.slot = slot;
  return cuda_ok(idx::launch_write_kv(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t idx_tree_state_size(const idx_tree_problem *problem, int32_t sel_k) {
  if (check_problem(problem, sel_k) != IDX_OK) return 0;
  return state_layout(problem, sel_k).total;
}

idx_status idx_tree_attention(const idx_tree_problem *problem, void *out, float *lse, void *state, size_t state_bytes,
                              void *stream) {
  return attend(problem, nullptr, 0, out, lse, state, state_bytes, stream);
}

idx_status idx_tree_attention_selected(const idx_tree_problem *problem, const int32_t *sel, int32_t sel_k, void *out,
                                       float *lse, void *state, size_t state_bytes, void *stream) {
  if (sel == nullptr || sel_k < 1) return IDX_EINVAL;
  return attend(problem, sel, sel_k, out, lse, state, state_bytes, stream);
}

}  // extern "C"
