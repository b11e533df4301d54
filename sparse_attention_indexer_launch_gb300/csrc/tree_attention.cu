// Attention of drafted tokens over a paged cache, whole or at selected positions.
//
// For a key/value head the query vectors that read it (tokens x query heads per
// key/value head) are the M = 128 rows of a tensor-core tile, and 128 cache
// positions (two pages) its columns:
//
//     S = Q K^T (TMEM)  ->  P = exp2(c S - m), rows' running maximum m and sum l
//                       ->  O += P V (TMEM, P read back from TMEM as operand A)
//
// K comes from shared memory with its dimensions contiguous, V as the transposed
// (MN-major) operand straight from the same page layout, so neither is rearranged.
//
// Work: an item is (request, key/value head, block of tokens) with its tiles in
// position order; the launch's tiles, in item order, are dealt out as one even,
// contiguous share per CTA (one CTA per SM).  A CTA that holds a whole item writes
// its output; shares of an item go to the state as (O, m, l) and the combine kernel
// joins them in CTA order, so equal calls give equal bits.
//
// Two streams hide the softmax behind the tensor core: the streams are either the
// even and odd tiles of one row block (up to 128 rows, joined in TMEM at the end of
// the item: more bytes in flight for the few-row, memory-bound calls) or two row
// blocks over the same tiles (more rows: each K and V tile is read from shared
// memory for 256 rows).  Each has S and O in 2 x 128 of TMEM's 512 columns, its own
// MMA-issuing thread and its own four softmax warps, one thread per row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "idx_device.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr int kTile = 128;               // keys per tile
constexpr int kRows = 128;               // rows of a stream
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // + 128 * stream
constexpr int kMinTiles = 2;             // tiles per CTA, at least (fewer CTAs otherwise)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's maximum moves only when a score passes it by 2^8: until then the sums run
// on the old one, below 2^8 * 2^19 in fp32, and O needs no pass through registers.
constexpr float kLazy = 8.0f;

// ---------------------------------------------------------------------------- roles
// warps 0-3 and 4-7: softmax of streams 0 and 1; 8: TMA producer; 9 and 10: MMA
// issuers of streams 0 and 1; 11: idle (keeps the loaders warpgroup-aligned);
// 12 ..: E4M3 to bf16 (four warps), or the gathering loaders (eight: K, V).
constexpr int kProducerWarp = 8, kIssuerWarp = 9, kLoaderWarp = 12;

template <int D, bool F8, bool PAIR, bool SEL>
struct Cfg {
  static constexpr int kTileBytes = kTile * D * 2;       // a K or V tile as bf16
  static constexpr int kRawBytes = kTile * D;            // ... as E4M3 bytes
  static constexpr bool kConvert = F8 && !SEL;           // raw tiles by TMA, then conversion
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kQBufs = PAIR || kConvert ? 1 : 2;
  static constexpr int kQTotal = kQBytes * (PAIR ? 2 : kQBufs);
  // bf16: 128 KB of tiles; E4M3: 80 KB (48 KB beside two row blocks) of raw tiles and
  // 96 KB of converted ones
  static constexpr int kStages = kConvert ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
  static constexpr int kRawStages = kConvert ? (D == 128 ? (PAIR ? 3 : 5) : 6) : 0;
  static constexpr int kScaleStages = F8 ? 8 : 0;
  static constexpr int kLoaderWarps = SEL ? 8 : kConvert ? 4 : 0;
  static constexpr int kThreads = 32 * (kLoaderWarps ? kLoaderWarp + kLoaderWarps : kLoaderWarp);
  static constexpr int kDynamic =
      1024 + kQTotal + kStages * kTileBytes + kRawStages * kRawBytes + kScaleStages * 2 * kTile * 4;
};

struct Barriers {
  uint64_t kv_full[8], kv_empty[8];
  uint64_t raw_full[6], raw_empty[6];
  uint64_t sc_full[8], sc_empty[8];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_ready[2], pv_done[2], o_free[2], drain[2], stats[2];
  int64_t start_base, total;       // tiles before the first request of the share, of the launch
  int32_t start_req;
  uint32_t tmem_base;
  int abort;
  int32_t two_terms[2];            // the stream's P has a low term
  uint32_t pages_ok[16];           // dense: bit h: page h of the CTA's tile k % 16 was loaded
  uint32_t keys_ok[16][4];         // selected: bit per key of tile k % 16
  int32_t nonfinite[8];            // segment number + 1 whose drafted tokens' V held NaN or infinity
  float row_m[2][2][kRows], row_l[2][2][kRows];   // [segment parity][stream][row]
  int64_t warp_sums[20];
};

// ---------------------------------------------------------------------------- TMEM
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void reg_fence32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
      "%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D += A B with A in TMEM (one 32-bit column holds two consecutive K elements of a row).
__device__ __forceinline__ void umma_f16_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// Descriptor of an MN-major operand in the 128-byte swizzle: 64 elements of the M or N
// dimension contiguous, groups of eight K rows 1024 bytes apart, the next 64 elements
// `block` bytes on.
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t smem_addr, uint32_t block) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((block >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
constexpr uint32_t kIdescBMn = 1u << 16;   // operand B is MN-major

__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z, int w, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four E4M3 codes to four bf16 values (exact: every E4M3 value is one).
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t x) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x >> 16), __NV_E4M3);
  const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
  return make_uint2(pack_bf16(fa.x, fa.y), pack_bf16(fb.x, fb.y));
}

// ---------------------------------------------------------------------------- plan
// A request as the launch reads it, clamped to the host's bounds.
struct Req {
  int32_t row0;    // first row
  int32_t tokens;  // drafted tokens
  int32_t ctx;     // cached tokens
  int32_t keys;    // ctx + tokens, within the page table
  int32_t tiles;   // of one item
  int32_t blocks;  // items per key/value head
  uint32_t bad;
};

template <bool SEL>
__device__ __forceinline__ Req load_req(const TreeAttnArgs &a, int i) {
  const idx_tree_problem &p = a.p;
  Req q;
  q.bad = 0;
  const int32_t r0 = p.row_start[i], r1 = p.row_start[i + 1];
  int32_t ctx = p.ctx_len[i];
  q.row0 = r0;
  q.tokens = 0;
  if (r0 < 0 || r1 > p.R || r1 < r0) q.bad = kStatusBadBound;
  else q.tokens = r1 - r0;
  if (q.tokens > p.max_new) {
    q.bad = kStatusBadBound;
    q.tokens = p.max_new;
  }
  if (ctx < 0 || ctx > p.max_ctx) q.bad = kStatusBadBound;
  ctx = max(0, min(ctx, p.max_ctx));
  q.ctx = ctx;
  const int64_t room = static_cast<int64_t>(p.pt_stride) * kPage;
  int64_t keys = static_cast<int64_t>(ctx) + q.tokens;
  if (keys > room) {
    q.bad = kStatusBadBound;
    keys = room;
  }
  q.keys = static_cast<int32_t>(keys);
  const int64_t n = SEL ? static_cast<int64_t>(a.sel_k) + q.tokens : keys;
  q.tiles = q.tokens > 0 ? static_cast<int32_t>((n + kTile - 1) / kTile) : 0;
  q.blocks = (q.tokens + a.item_tokens - 1) / a.item_tokens;
  return q;
}
__device__ __forceinline__ int64_t req_tiles(const Req &q, int hkv) {
  return static_cast<int64_t>(q.tiles) * q.blocks * hkv;
}
// Shares: CTA c of n takes tiles [c W / n, (c + 1) W / n).
__device__ __forceinline__ int64_t share_begin(int64_t W, int n, int c) { return W * c / n; }
__device__ __forceinline__ int share_count(int64_t W, int ctas) {
  const int64_t n = (W + kMinTiles - 1) / kMinTiles;
  return n < 1 ? 1 : n > ctas ? ctas : static_cast<int>(n);
}

// Walks the segments of a share: the tiles of one item that fall into it.
template <bool SEL>
struct Walk {
  const TreeAttnArgs &a;
  int64_t t, end, base;   // next tile, end of the share, tiles before request i
  int i;
  Req q;
  // the segment
  int seg = -1;           // its number
  int head, tok0, tokens; // key/value head; first token and token count of the item's block
  int tile0, count;       // first tile within the item, tiles
  bool whole;             // the segment is the whole item
  bool first;             // it is the share's first segment (its partial goes to slot 0)
  int64_t share0;

  __device__ __forceinline__ Walk(const TreeAttnArgs &args, int64_t t0, int64_t t1, int req, int64_t req_base)
      : a(args), t(t0), end(t1), base(req_base), i(req), share0(t0) {
    if (t < end) q = load_req<SEL>(a, i);
  }
  __device__ __forceinline__ bool next() {
    if (t >= end) return false;
    int64_t mine = req_tiles(q, a.p.cache.Hkv);
    while (t >= base + mine) {
      base += mine;
      q = load_req<SEL>(a, ++i);
      mine = req_tiles(q, a.p.cache.Hkv);
    }
    const int64_t off = t - base;
    const int64_t item = off / q.tiles;
    tile0 = static_cast<int>(off - item * q.tiles);
    head = static_cast<int>(item / q.blocks);
    const int block = static_cast<int>(item - static_cast<int64_t>(head) * q.blocks);
    tok0 = block * a.item_tokens;
    tokens = min(a.item_tokens, q.tokens - tok0);
    const int64_t left = end - t;
    count = static_cast<int>(min(left, static_cast<int64_t>(q.tiles - tile0)));
    whole = tile0 == 0 && count == q.tiles;
    first = t == share0;
    t += count;
    ++seg;
    return true;
  }
};

// Place of tile j's K and V in the order K0 K1 V0 K2 V1 ... of a segment of n tiles.
__device__ __forceinline__ int pos_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int pos_v(int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * n - 1; }

// ---------------------------------------------------------------------------- softmax
// One row of a tile: S (128 columns at ts) to P in the same columns, the row's maximum m
// and sum l, and O (D columns at to) when the maximum moves.  kPartial: only the keys of
// okbits are visible.
//
// P is rounded to bf16 for the product with V.  Over the 128 or more keys of a full tile
// the roundings average out below the output's own; the few keys of a partial tile do
// not, so there P is kept in two bf16 terms, high in columns 0-63 and low in 64-127, and
// the product runs over both.
template <int D, bool F8, bool kPartial>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t to, const float4 *sc, float c,
                                             const uint32_t (&okbits)[4], bool has_o, float &m, float &l) {
  auto visible = [&](int w, int y) { return !kPartial || ((okbits[w] >> y) & 1u); };
  // the row's maximum, in units of log2
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t x[32];
    tmem_ld32(ts + 32 * w, x);
    tmem_wait_ld();
    reg_fence32(x);
#pragma unroll
    for (int y = 0; y < 32; y += 4) {
      const float4 ks = F8 ? sc[8 * w + (y >> 2)] : make_float4(1.f, 1.f, 1.f, 1.f);
      const float kk[4] = {ks.x, ks.y, ks.z, ks.w};
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const float v = F8 ? __uint_as_float(x[y + z]) * kk[z] : __uint_as_float(x[y + z]);
        top = visible(w, y + z) ? fmaxf(top, v) : top;
      }
    }
  }
  top *= c;
  if (top != top) top = 0.0f;   // scale 0: 0 x -inf moves no maximum
  const bool grow = top > m + kLazy || (m == -INFINITY && top > -INFINITY);
  if (__any_sync(0xffffffffu, grow)) {
    const float nm = fmaxf(m, top);
    const float f = m == -INFINITY ? 0.0f : ex2(m - nm);
    m = nm;
    l *= f;
    if (has_o) {
#pragma unroll 1
      for (int w = 0; w < D / 32; ++w) {
        uint32_t x[32];
        tmem_ld32(to + 32 * w, x);
        tmem_wait_ld();
        reg_fence32(x);
#pragma unroll
        for (int y = 0; y < 32; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * f);
        tmem_st32(to + 32 * w, x);
      }
    }
  }
  const float base = m == -INFINITY ? 0.0f : m;
  float l0 = 0.0f, l1 = 0.0f;
  uint32_t low[kPartial ? 2 : 1][16];   // low terms whose columns S still holds
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t x[32], hi[16], lo[16];
    tmem_ld32(ts + 32 * w, x);
    tmem_wait_ld();
    reg_fence32(x);
#pragma unroll
    for (int y = 0; y < 32; y += 4) {
      const float4 ks = F8 ? sc[8 * w + (y >> 2)] : make_float4(1.f, 1.f, 1.f, 1.f);
      const float4 vs = F8 ? sc[32 + 8 * w + (y >> 2)] : make_float4(1.f, 1.f, 1.f, 1.f);
      const float kk[4] = {ks.x, ks.y, ks.z, ks.w}, vv[4] = {vs.x, vs.y, vs.z, vs.w};
      float e[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const float v = F8 ? __uint_as_float(x[y + z]) * kk[z] : __uint_as_float(x[y + z]);
        e[z] = ex2(fmaf(v, c, -base));
        if (!visible(w, y + z)) e[z] = 0.0f;
        (z & 1 ? l1 : l0) += e[z];
        if (F8) {
          e[z] *= vv[z];
          if (!visible(w, y + z)) e[z] = 0.0f;   // a stale scale may be NaN
        }
      }
#pragma unroll
      for (int z = 0; z < 4; z += 2) {
        const uint32_t h = pack_bf16(e[z], e[z + 1]);
        hi[(y + z) >> 1] = h;
        if (kPartial) {
          // an infinity (a scale's) has no low term
          const float r0 = e[z] - __uint_as_float(h << 16), r1 = e[z + 1] - __uint_as_float(h & 0xFFFF0000u);
          lo[(y + z) >> 1] = pack_bf16(r0 == r0 ? r0 : 0.0f, r1 == r1 ? r1 : 0.0f);
        }
      }
    }
    tmem_st16(ts + 16 * w, hi);
    if (kPartial) {
      // columns 64-95 are free once chunk 2 is read, 96-127 once chunk 3 is
      constexpr int kLast = kPartial ? 1 : 0;
      if (w == 2) {
        tmem_st16(ts + 64, low[0]);
        tmem_st16(ts + 80, low[kLast]);
      }
      if (w == 3) {
        tmem_st16(ts + 96, low[0]);
        tmem_st16(ts + 112, lo);
      } else {
#pragma unroll
        for (int y = 0; y < 16; ++y) low[w == 1 ? kLast : 0][y] = lo[y];
      }
    }
    (void)lo;
  }
  l += l0 + l1;
  tmem_wait_st();
}

// ---------------------------------------------------------------------------- kernel
template <int D, bool F8, bool PAIR, bool SEL>
__global__ void __launch_bounds__(Cfg<D, F8, PAIR, SEL>::kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const TreeAttnArgs a) {
  using C = Cfg<D, F8, PAIR, SEL>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Barriers bars;
  uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  uint8_t *const sq = smem;
  uint8_t *const skv = sq + C::kQTotal;
  uint8_t *const sraw = skv + C::kStages * C::kTileBytes;
  float *const ssc = reinterpret_cast<float *>(sraw + C::kRawStages * C::kRawBytes);   // [stage][K 128, V 128]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const idx_tree_problem &p = a.p;
  const int Hkv = p.cache.Hkv;
  const int G = p.Hq / Hkv;
  constexpr int kBlocks = D / 64;            // 64-dimension blocks of an operand tile
  constexpr int kBlockBytes = kTile * 128;
  grid_dependency_trigger();                 // the combine kernel's CTAs may take free SMs

  if (tid == 0) {
    for (int s = 0; s < 8; ++s) {
      // filled by one TMA thread, by the 128 converting threads, or by a gathering team
      mbar_init(&bars.kv_full[s], SEL || C::kConvert ? 128 : 1);
      mbar_init(&bars.kv_empty[s], PAIR ? 2 : 1);
      mbar_init(&bars.sc_full[s], SEL ? 256 : 1);
      mbar_init(&bars.sc_empty[s], PAIR ? 256 : 128);
    }
    for (int s = 0; s < 6; ++s) {
      mbar_init(&bars.raw_full[s], 1);
      mbar_init(&bars.raw_empty[s], 128);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.q_full[s], 1);
      mbar_init(&bars.q_empty[s], 2);
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.p_ready[s], 128);
      mbar_init(&bars.pv_done[s], 1);
      mbar_init(&bars.o_free[s], PAIR ? 128 : 256);
      mbar_init(&bars.drain[s], 1);
      mbar_init(&bars.stats[s], 128);
    }
    bars.abort = 0;
    for (int s = 0; s < 8; ++s) bars.nonfinite[s] = 0;
    fence_barrier_init();
  }
  if (warp == kIssuerWarp) {
    tmem_alloc(&bars.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (tid == kProducerWarp * 32) {
    prefetch_tensormap(&qmap);
    if (!SEL) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
  }

  // ------------------------------------------------------------------ the share
  // Every CTA sums the requests' tiles itself; CTA 0 keeps the prefix sums for the
  // combine kernel.
  constexpr int kWarps = C::kThreads / 32;
  int64_t W = 0;
  {
    uint32_t bad = 0;
    int64_t mine = 0, incl = 0;
    auto scan = [&](int i0, int64_t before) -> int64_t {   // inclusive sums of one chunk, returns its total
      const int i = i0 + tid;
      mine = 0;
      if (i < p.Q) {
        const Req q = load_req<SEL>(a, i);
        bad |= q.bad;
        mine = req_tiles(q, Hkv);
      }
      incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) bars.warp_sums[warp] = incl;
      __syncthreads();
      int64_t total = 0;
      incl += before;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += bars.warp_sums[w];
        total += bars.warp_sums[w];
      }
      __syncthreads();
      return total;
    };
    for (int i0 = 0; i0 < p.Q; i0 += C::kThreads) {
      const int64_t before = W;
      W += scan(i0, before);
      if (blockIdx.x == 0 && i0 + tid < p.Q) a.prefix[i0 + tid] = incl - mine;
    }
    if (blockIdx.x == 0) {
      if (tid == 0) a.prefix[p.Q] = W;
      if (bad) flag_status(a.status, bad);
    }
    const int n = share_count(W, gridDim.x);
    const int64_t t0 = static_cast<int>(blockIdx.x) < n ? share_begin(W, n, blockIdx.x) : W;
    if (t0 < W) {
      int64_t before = 0;
      for (int i0 = 0; i0 < p.Q; i0 += C::kThreads) {
        if (p.Q > C::kThreads) before += scan(i0, before);   // one chunk: the sums are still in registers
        if (i0 + tid < p.Q && t0 >= incl - mine && t0 < incl) {
          bars.start_req = i0 + tid;
          bars.start_base = incl - mine;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const int nshare = share_count(W, gridDim.x);
  const bool idle = static_cast<int>(blockIdx.x) >= nshare;
  const int64_t t0 = idle ? 0 : share_begin(W, nshare, blockIdx.x);
  const int64_t t1 = idle ? 0 : share_begin(W, nshare, blockIdx.x + 1);
  const int req0 = t0 < t1 ? bars.start_req : 0;
  const int64_t base0 = t0 < t1 ? bars.start_base : 0;
  Walk<SEL> walk(a, t0, t1, req0, base0);

  const uint64_t limit = a.wait_limit_ns;
  volatile int *abort = &bars.abort;
  int never = 0;
  // A wait whose outcome the whole warp shares (so that it leaves its loop together).
  auto warp_wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
    const bool r = mbar_wait(bar, parity, limit, abort);
    return __all_sync(0xffffffffu, r);
  };
  auto give_up = [&]() {
    flag_status(a.status, kStatusTimeout);
    *abort = 1;
  };

  if (warp == kProducerWarp) {
    // ---------------------------------------------------------------- producer
    int nload = 0;      // K and V tiles so far
    int nscale = 0;     // tiles with scales so far
    int nq = 0;         // Q loads so far
    bool ok = true;
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
      int r = 1;
      if (lane == 0) r = mbar_wait(bar, parity, limit, abort);
      return __shfl_sync(0xffffffffu, r, 0) != 0;
    };
    while (ok && walk.next()) {
      // Q of the segment
      const int qb = walk.seg % C::kQBufs;
      if (!warp_wait(&bars.q_empty[qb], ((walk.seg / C::kQBufs) & 1) ^ 1)) {
        ok = false;
        break;
      }
      const int tb = PAIR ? a.item_tokens / 2 : a.item_tokens;   // tokens of a stream's rows
      if (lane == 0) {
        const int nhalf = PAIR && walk.tokens > tb ? 2 : 1;
        mbar_arrive_expect_tx(&bars.q_full[qb], static_cast<uint32_t>(nhalf * kBlocks * G * tb * 128));
        for (int s = 0; s < nhalf; ++s)
          for (int b = 0; b < kBlocks; ++b)
            tma_load_3d(sq + (PAIR ? s : qb) * C::kQBytes + b * kBlockBytes, &qmap, b * 64, walk.head * G,
                        walk.q.row0 + walk.tok0 + s * tb, &bars.q_full[qb]);
      }
      ++nq;
      if (SEL) continue;   // K and V are gathered by the loaders
      const int npages = (walk.q.keys + kPage - 1) / kPage;
      const int32_t *const table = p.page_table + static_cast<int64_t>(walk.i) * p.pt_stride;
      int32_t ids = -2, ids_next = -2;
      auto fetch = [&](int j0) -> int32_t {   // page ids of tiles j0 .. j0 + 15 of the segment (-2: none)
        const int pg = (walk.tile0 + j0) * 2 + lane;
        return pg < npages ? table[pg] : -2;
      };
      ids = fetch(0);
      int32_t vids0 = -1, vids1 = -1;   // pages of tile j - 1, whose V follows K of tile j
      for (int j = 0; ok && j <= walk.count; ++j) {
        int32_t pg[2] = {-1, -1};
        if (j < walk.count) {
          if ((j & 15) == 0) {
            if (j > 0) ids = ids_next;
            ids_next = fetch(j + 16);
          }
          pg[0] = __shfl_sync(0xffffffffu, ids, (j & 15) * 2);
          pg[1] = __shfl_sync(0xffffffffu, ids, (j & 15) * 2 + 1);
          uint32_t flags = 0;
          for (int h = 0; h < 2; ++h) {
            if (pg[h] >= 0 && pg[h] < p.cache.P) {
              flags |= 1u << h;
            } else {
              if (pg[h] != -2 && lane == 0) flag_status(a.status, kStatusBadPage);
              pg[h] = -1;
            }
          }
          if (lane == 0) bars.pages_ok[nscale & 15] = flags;
        }
        // K of tile j, then V of tile j - 1
        for (int what = 0; what < 2; ++what) {
          if (what == 0 ? j >= walk.count : j == 0) continue;
          const int32_t g0 = what == 0 ? pg[0] : vids0, g1 = what == 0 ? pg[1] : vids1;
          const uint32_t npg = (g0 >= 0) + (g1 >= 0);
          uint8_t *dst;
          uint64_t *full;
          if constexpr (C::kConvert) {
            const int s = nload % C::kRawStages;
            if (!warp_wait(&bars.raw_empty[s], ((nload / C::kRawStages) & 1) ^ 1)) {
              ok = false;
              break;
            }
            dst = sraw + s * C::kRawBytes;
            full = &bars.raw_full[s];
          } else {
            const int s = nload % C::kStages;
            if (!warp_wait(&bars.kv_empty[s], ((nload / C::kStages) & 1) ^ 1)) {
              ok = false;
              break;
            }
            dst = skv + s * C::kTileBytes;
            full = &bars.kv_full[s];
          }
          if (F8 && what == 0) {
            const int s = nscale % 8;
            if (!warp_wait(&bars.sc_empty[s], ((nscale / 8) & 1) ^ 1)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(&bars.sc_full[s], npg * 512u);
              float *const d = ssc + s * 2 * kTile;
              for (int h = 0; h < 2; ++h) {
                if (pg[h] < 0) continue;
                const int64_t at = (static_cast<int64_t>(pg[h]) * Hkv + walk.head) * kPage;
                bulk_load(d + h * kPage, p.cache.k_scale + at, 256u, &bars.sc_full[s]);
                bulk_load(d + kTile + h * kPage, p.cache.v_scale + at, 256u, &bars.sc_full[s]);
              }
            }
          }
          if (lane == 0) {
            const void *const map = what == 0 ? &kmap : &vmap;
            mbar_arrive_expect_tx(full, npg * static_cast<uint32_t>(F8 ? kPage * D : kPage * D * 2));
            for (int h = 0; h < 2; ++h) {
              const int32_t g = h == 0 ? g0 : g1;
              if (g < 0) continue;
              if constexpr (F8) {
                tma_load_4d(dst + h * kPage * D, map, 0, 0, walk.head, g, full);
              } else {
                for (int b = 0; b < kBlocks; ++b)
                  tma_load_4d(dst + b * kBlockBytes + h * kPage * 128, map, b * 64, 0, walk.head, g, full);
              }
            }
          }
          ++nload;
          if (what == 0) ++nscale;
        }
        vids0 = pg[0];
        vids1 = pg[1];
      }
    }
    if (!ok && lane == 0) give_up();
    // every copy still in flight lands before the CTA may exit (also after giving up)
    if (lane == 0) {
      auto land = [&](uint64_t *bar, int n, int used) {
        for (int s = 0; s < n; ++s) {
          if (used <= s) continue;
          const int last = used - 1 - (used - 1 - s) % n;
          if (!mbar_wait(&bar[s], (last / n) & 1, limit, &never)) flag_status(a.status, kStatusTimeout);
        }
      };
      land(bars.q_full, C::kQBufs, nq);
      if constexpr (C::kConvert) land(bars.raw_full, C::kRawStages, nload);
      else if (!SEL) land(bars.kv_full, C::kStages, nload);
      if (F8 && !SEL) land(bars.sc_full, 8, nscale);
    }
  } else if (warp == kIssuerWarp || warp == kIssuerWarp + 1) {
    // ---------------------------------------------------------------- MMA issuers
    // Per stream: S of a tile, then (its P ready) O += P V, then the next S once that
    // has completed, since P lies in S's columns; the other stream's MMAs fill the gap.
    if (lane == 0) {
      const int s = warp - kIssuerWarp;
      const uint32_t ts = tmem + kColS + 128 * s, to = tmem + kColO + 128 * s;
      const uint32_t idesc_s = umma_idesc(1u, kTile), idesc_o = umma_idesc(1u, D) | kIdescBMn;
      int loads = 0;      // K and V tiles of earlier segments
      uint32_t n = 0;     // this stream's tiles so far
      bool ok = true, any = false;
      while (ok && walk.next()) {
        const int qb = walk.seg % C::kQBufs;
        const bool live = !PAIR || s == 0 || walk.tokens > a.item_tokens / 2;   // this stream has rows
        if (!mbar_wait(&bars.q_full[qb], (walk.seg / C::kQBufs) & 1, limit, abort)) {
          ok = false;
          break;
        }
        const uint64_t qdesc = umma_desc_sw128(smem_u32(sq + (PAIR ? s : qb) * C::kQBytes));
        const int step = PAIR ? 1 : 2, j0 = PAIR ? 0 : s;
        if (j0 >= walk.count) mbar_arrive(&bars.q_empty[qb]);
        for (int j = j0; j < walk.count; j += step) {
          const int lk = loads + pos_k(j), lv = loads + pos_v(j, walk.count);
          const int sk = lk % C::kStages, sv = lv % C::kStages;
          if (!mbar_wait(&bars.kv_full[sk], (lk / C::kStages) & 1, limit, abort)) {
            ok = false;
            break;
          }
          if (!live) {   // no rows: only pass the tiles on
            mbar_arrive(&bars.kv_empty[sk]);
            if (j + step >= walk.count) mbar_arrive(&bars.q_empty[qb]);
            if (!mbar_wait(&bars.kv_full[sv], (lv / C::kStages) & 1, limit, abort)) {
              ok = false;
              break;
            }
            mbar_arrive(&bars.kv_empty[sv]);
            continue;
          }
          tc_fence_after();
          const uint64_t kdesc = umma_desc_sw128(smem_u32(skv + sk * C::kTileBytes));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kBlockBytes + (kk & 3) * 32) >> 4;
            umma_f16(ts, qdesc + off, kdesc + off, idesc_s, kk > 0);
          }
          umma_commit(&bars.kv_empty[sk]);
          umma_commit(&bars.s_full[s]);
          if (j + step >= walk.count) umma_commit(&bars.q_empty[qb]);
          any = true;
          if (!mbar_wait(&bars.p_ready[s], n & 1, limit, abort) ||
              (j == j0 && !mbar_wait(&bars.o_free[s], (walk.seg & 1) ^ 1, limit, abort)) ||
              !mbar_wait(&bars.kv_full[sv], (lv / C::kStages) & 1, limit, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t vdesc = umma_desc_mn(smem_u32(skv + sv * C::kTileBytes), kBlockBytes);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            umma_f16_ta(to, ts + kk * 8, vdesc + ((kk * 2048) >> 4), idesc_o, j > j0 || kk > 0);
          if (*reinterpret_cast<volatile int32_t *>(&bars.two_terms[s])) {
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_f16_ta(to, ts + 64 + kk * 8, vdesc + ((kk * 2048) >> 4), idesc_o, 1u);
          }
          umma_commit(&bars.kv_empty[sv]);
          umma_commit(&bars.pv_done[s]);
          if (!mbar_wait(&bars.pv_done[s], n & 1, limit, abort)) {
            ok = false;
            break;
          }
          ++n;
        }
        loads += 2 * walk.count;
      }
      if (!ok) {
        give_up();
        if (any) {   // MMAs in flight read shared memory and TMEM: wait for them
          umma_commit(&bars.drain[s]);
          if (!mbar_wait(&bars.drain[s], 0, limit, &never)) flag_status(a.status, kStatusTimeout);
        }
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int s = warp >> 2;               // stream
    const int row = tid & 127;             // row of the stream's tile, and its TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // first TMEM lane of the warp << 16
    const uint32_t ts = tmem + kColS + 128 * s + lanes;
    const uint32_t to = tmem + kColO + 128 * s + lanes;
    const float c = p.scale * kLog2e;
    const int step = PAIR ? 1 : 2, j0 = PAIR ? 0 : s;
    int tiles = 0;      // tiles of earlier segments
    uint32_t n = 0;     // this stream's tiles so far
    bool ok = true;
    while (ok && walk.next()) {
      const int tb = PAIR ? a.item_tokens / 2 : a.item_tokens;
      const int stok0 = walk.tok0 + (PAIR ? s * tb : 0);                       // first token of the stream
      const int nrow = max(0, min(tb, walk.tokens - (PAIR ? s * tb : 0))) * G; // its rows
      const bool live = !PAIR || nrow > 0;                                     // the issuer runs it
      const bool active = (row & ~31) < nrow;                                  // the warp has rows
      const int tok = min(stok0 + row / G, walk.q.tokens - 1);
      const int r = walk.q.row0 + tok;
      uint64_t mask = 0;
      if (row < nrow) mask = p.mask != nullptr ? p.mask[r] : (2ull << tok) - 1ull;
      const int ctx = walk.q.ctx;
      float m = -INFINITY, l = 0.0f;
      int mine = 0;      // this stream's tiles in the segment
      for (int j = j0; live && j < walk.count; j += step, ++n, ++mine) {
        const int k = tiles + j;
        const int key0 = (walk.tile0 + j) * kTile;
        if (F8 && !warp_wait_all(&bars.sc_full[k % 8], (k / 8) & 1)) {
          ok = false;
          break;
        }
        if (!warp_wait_all(&bars.s_full[s], n & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t okbits[4] = {~0u, ~0u, ~0u, ~0u};   // keys of the tile that the row sees
        bool special;
        if (SEL) {
          special = false;
          for (int w = 0; w < 4; ++w) {
            okbits[w] = bars.keys_ok[k & 15][w];
            special |= okbits[w] != ~0u;
          }
        } else {
          const uint32_t flags = bars.pages_ok[k & 15];
          special = key0 + kTile > ctx || flags != 3u;
          if (special) {
            const int lim = walk.q.keys - ctx;      // drafted tokens within the page table
            const uint64_t vm = lim >= 64 ? mask : mask & ((1ull << lim) - 1ull);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int before = ctx - (key0 + 32 * w);   // cached keys from the word's first on
              uint32_t bits;
              if (before >= 32) bits = ~0u;
              else if (before > 0) bits = ((1u << before) - 1u) | static_cast<uint32_t>(vm << before);
              else bits = before > -64 ? static_cast<uint32_t>(vm >> -before) : 0u;
              okbits[w] = (flags >> (w >> 1)) & 1u ? bits : 0u;
            }
          }
        }
        if (!SEL && !C::kConvert && special) {
          // V of tokens that some rows do not see has to be finite (0 x NaN is NaN): zero
          // what no row sees, and what is not finite among the drafted tokens (rows that
          // see it get it back at the end)
          const int lv = 2 * tiles + pos_v(j, walk.count);
          const int sv = lv % C::kStages;
          if (!warp_wait_all(&bars.kv_full[sv], (lv / C::kStages) & 1)) {
            ok = false;
            break;
          }
          const int pos = key0 + row;
          const bool dead = pos >= walk.q.keys || !((bars.pages_ok[k & 15] >> (row >> 6)) & 1u);
          if (dead || pos >= ctx) {
#pragma unroll
            for (int x = 0; x < kBlocks * 8; ++x) {
              uint4 *const at = reinterpret_cast<uint4 *>(skv + sv * C::kTileBytes + (x >> 3) * kBlockBytes + row * 128 +
                                                          ((x + row) & 7) * 16);
              uint4 v = dead ? make_uint4(0, 0, 0, 0) : *at;
              if (!dead) {
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
                bool changed = false;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  if ((w[y] & 0x7F80u) == 0x7F80u) { w[y] &= 0xFFFF0000u; changed = true; }
                  if ((w[y] & 0x7F800000u) == 0x7F800000u) { w[y] &= 0xFFFFu; changed = true; }
                }
                if (!changed) continue;
                bars.nonfinite[walk.seg & 7] = walk.seg + 1;
                v = make_uint4(w[0], w[1], w[2], w[3]);
              }
              *at = v;
            }
          }
          fence_proxy_async_shared();
        }
        if (active) {
          const float4 *const sc = reinterpret_cast<const float4 *>(ssc + (k % 8) * 2 * kTile);
          if (special) softmax_tile<D, F8, true>(ts, to, sc, c, okbits, mine > 0, m, l);
          else softmax_tile<D, F8, false>(ts, to, sc, c, okbits, mine > 0, m, l);
        }
        if (row == 0) bars.two_terms[s] = special;
        tc_fence_before();
        mbar_arrive(&bars.p_ready[s]);
        if (F8) mbar_arrive(&bars.sc_empty[k % 8]);
      }
      if (!ok) break;
      if (F8 && PAIR && !live)   // hand the scales of the tiles on
        for (int j = 0; j < walk.count; ++j) {
          const int k = tiles + j;
          if (!warp_wait_all(&bars.sc_full[k % 8], (k / 8) & 1)) {
            ok = false;
            break;
          }
          mbar_arrive(&bars.sc_empty[k % 8]);
        }
      if (!ok) break;
      tiles += walk.count;

      // -------------------------------------------------------------- end of the segment
      if (mine > 0 && !warp_wait_all(&bars.pv_done[s], (n - 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (l != l) m = INFINITY;   // a NaN among the visible scores takes the whole row, in every join
      float f0 = 1.0f, f1 = 0.0f;
      int d0 = 0, dn = D;     // the columns that this thread writes
      if (!PAIR) {
        // join the streams: both sides get the common maximum, each writes half of O
        const int sp = walk.seg & 1;
        bars.row_m[sp][s][row] = m;
        bars.row_l[sp][s][row] = l;
        tc_fence_before();
        mbar_arrive(&bars.stats[s]);
        if (!warp_wait_all(&bars.stats[s ^ 1], walk.seg & 1)) {
          ok = false;
          break;
        }
        const float m0 = bars.row_m[sp][0][row], m1 = bars.row_m[sp][1][row];
        const float mm = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.0f : ex2(m0 - mm);
        f1 = m1 == -INFINITY ? 0.0f : ex2(m1 - mm);
        l = bars.row_l[sp][0][row] * f0 + bars.row_l[sp][1][row] * f1;
        m = mm;
        d0 = s * (D / 2);
        dn = D / 2;
      }
      tc_fence_after();
      const bool two = !PAIR && walk.count > 1;    // stream 1 has tiles
      const bool poison = *reinterpret_cast<volatile int32_t *>(&bars.nonfinite[walk.seg & 7]) == walk.seg + 1;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int hq = walk.head * G + row % G;
      const int slot = (walk.first ? 0 : 1) + 2 * static_cast<int>(blockIdx.x);
      const int prow = (PAIR ? s * kRows : 0) + row;
      constexpr int kSlotRows = PAIR ? 2 * kRows : kRows;
      if (active) {
        for (int d = d0; d < d0 + dn; d += 32) {
          uint32_t x[32];
          const uint32_t o0 = PAIR ? to : tmem + kColO + lanes;
          __syncwarp();
          tmem_ld32(o0 + d, x);
          tmem_wait_ld();
          reg_fence32(x);
          float o[32];
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = PAIR ? __uint_as_float(x[y]) : f0 == 0.0f ? 0.0f : __uint_as_float(x[y]) * f0;
          if (two) {
            tmem_ld32(o0 + 128 + d, x);
            tmem_wait_ld();
            reg_fence32(x);
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] += f1 == 0.0f ? 0.0f : __uint_as_float(x[y]) * f1;
          }
          if (row < nrow) {
            if (l == 0.0f) {
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = 0.0f;
            }
            if (poison) {
              // what was zeroed for the rows that do not see it
              for (int u = 0; u < walk.q.tokens; ++u) {
                const int pos = ctx + u;
                if (!((mask >> u) & 1ull) || pos >= walk.q.keys || pos < walk.tile0 * kTile ||
                    pos >= (walk.tile0 + walk.count) * kTile)
                  continue;
                const int32_t pg = p.page_table[static_cast<int64_t>(walk.i) * p.pt_stride + pos / kPage];
                if (pg < 0 || pg >= p.cache.P) continue;
                const int64_t at = pg * p.cache.page_stride + (pos % kPage) * p.cache.token_stride +
                                   walk.head * p.cache.head_stride + d;
                for (int y = 0; y < 32; ++y) {
                  float v;
                  if (F8) v = static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(p.cache.v)[at + y]);
                  else v = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.cache.v)[at + y]);
                  if (!isfinite(v)) o[y] += v;
                }
              }
            }
            if (walk.whole) {
              uint16_t *const out = a.out + (static_cast<int64_t>(r) * p.Hq + hq) * D + d;
#pragma unroll
              for (int y = 0; y < 32; y += 8)
                *reinterpret_cast<uint4 *>(out + y) =
                    make_uint4(pack_bf16(o[y] * inv, o[y + 1] * inv), pack_bf16(o[y + 2] * inv, o[y + 3] * inv),
                               pack_bf16(o[y + 4] * inv, o[y + 5] * inv), pack_bf16(o[y + 6] * inv, o[y + 7] * inv));
            } else {
              float *const part = a.part_o + (static_cast<int64_t>(slot) * kSlotRows + prow) * D + d;
#pragma unroll
              for (int y = 0; y < 32; y += 4)
                *reinterpret_cast<float4 *>(part + y) = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
            }
          }
        }
        if (row < nrow && d0 == 0) {
          if (walk.whole) {
            if (a.lse != nullptr)
              a.lse[static_cast<int64_t>(r) * p.Hq + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
          } else {
            a.part_ml[static_cast<int64_t>(slot) * kSlotRows + prow] = make_float2(m, l);
          }
        }
      }
      tc_fence_before();
      if (PAIR) {
        mbar_arrive(&bars.o_free[s]);
      } else {
        mbar_arrive(&bars.o_free[0]);
        mbar_arrive(&bars.o_free[1]);
      }
    }
    if (!ok) give_up();
  } else if (warp >= kLoaderWarp) {
    if constexpr (C::kConvert) {
    // ---------------------------------------------------------------- E4M3 to bf16
    const int t = tid - kLoaderWarp * 32;
    int loads = 0, tiles = 0;
    bool ok = true;
    while (ok && walk.next()) {
      for (int x = 0; ok && x < 2 * walk.count; ++x, ++loads) {
        // place x of the segment is K of tile (x + 1) / 2 or V of tile x / 2 - 1
        const bool is_v = x == 2 * walk.count - 1 || (x > 0 && (x & 1) == 0);
        const int j = x == 2 * walk.count - 1 ? walk.count - 1 : is_v ? x / 2 - 1 : (x + 1) / 2;
        const int sr = loads % C::kRawStages, sk = loads % C::kStages;
        if (!warp_wait_all(&bars.raw_full[sr], (loads / C::kRawStages) & 1) ||
            !warp_wait_all(&bars.kv_empty[sk], ((loads / C::kStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        const uint8_t *const src = sraw + sr * C::kRawBytes;
        uint8_t *const dst = skv + sk * C::kTileBytes;
        const int key0 = (walk.tile0 + j) * kTile;
        const uint32_t flags = bars.pages_ok[(tiles + j) & 15];
        const bool special = is_v && (key0 + kTile > walk.q.ctx || flags != 3u);
        constexpr int kChunks = D / 16;     // 16-byte chunks of codes per key
#pragma unroll 4
        for (int y = t; y < kTile * kChunks; y += 128) {
          const int key = y / kChunks, ch = y % kChunks;
          uint4 v = *reinterpret_cast<const uint4 *>(src + key * D + ch * 16);
          if (special) {
            const int pos = key0 + key;
            if (pos >= walk.q.keys || !((flags >> (key >> 6)) & 1u)) {
              v = make_uint4(0, 0, 0, 0);
            } else if (pos >= walk.q.ctx) {
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
              for (int z = 0; z < 16; ++z) {
                if (((w[z >> 2] >> (8 * (z & 3))) & 0x7Fu) == 0x7Fu) {
                  w[z >> 2] &= ~(0xFFu << (8 * (z & 3)));
                  bars.nonfinite[walk.seg & 7] = walk.seg + 1;
                }
              }
              v = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          const uint2 a0 = e4m3x4_to_bf16(v.x), a1 = e4m3x4_to_bf16(v.y), a2 = e4m3x4_to_bf16(v.z),
                      a3 = e4m3x4_to_bf16(v.w);
          uint8_t *const row = dst + (ch >> 2) * kBlockBytes + key * 128;
          const int c0 = (ch & 3) * 2;
          *reinterpret_cast<uint4 *>(row + ((c0 ^ (key & 7)) << 4)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
          *reinterpret_cast<uint4 *>(row + (((c0 + 1) ^ (key & 7)) << 4)) = make_uint4(a2.x, a2.y, a3.x, a3.y);
        }
        fence_proxy_async_shared();
        mbar_arrive(&bars.kv_full[sk]);
        mbar_arrive(&bars.raw_empty[sr]);
      }
      tiles += walk.count;
    }
    if (!ok) give_up();
    } else if constexpr (SEL) {
    // ---------------------------------------------------------------- gathering loaders
    // Four warps bring K, four V.  A thread looks up one key of the tile; a group of
    // lanes then reads each key's D values with 16 bytes per lane.
    const int team = (warp - kLoaderWarp) >> 2;      // 0: K, 1: V
    const int t = (tid - kLoaderWarp * 32) & 127;    // key of the tile
    const int w4 = (warp - kLoaderWarp) & 3;
    int loads = 0, tiles = 0;
    bool ok = true;
    const uint8_t *const cache = static_cast<const uint8_t *>(team == 0 ? p.cache.k : p.cache.v);
    const float *const scales = team == 0 ? p.cache.k_scale : p.cache.v_scale;
    while (ok && walk.next()) {
      const int r = walk.q.row0 + walk.tok0;
      const uint64_t mask = p.mask != nullptr ? p.mask[r] : (2ull << walk.tok0) - 1ull;
      const int32_t *const sel = a.sel + static_cast<int64_t>(r) * a.sel_k;
      const int32_t *const table = p.page_table + static_cast<int64_t>(walk.i) * p.pt_stride;
      // page * 64 + token of the thread's key in tile j, or -1
      auto find = [&](int j) -> int32_t {
        const int n = (walk.tile0 + j) * kTile + t;
        int64_t pos = -1;
        if (n < a.sel_k) {
          const int32_t e = sel[n];
          if (e >= 0 && e < walk.q.ctx) pos = e;
        } else if (n < a.sel_k + walk.q.tokens) {
          const int u = n - a.sel_k;
          if ((mask >> u) & 1ull) pos = static_cast<int64_t>(walk.q.ctx) + u;
        }
        if (pos < 0 || pos >= walk.q.keys) return -1;
        const int32_t pg = table[pos / kPage];
        if (pg < 0 || pg >= p.cache.P) {
          if (team == 0) flag_status(a.status, kStatusBadPage);
          return -1;
        }
        return pg * kPage + static_cast<int32_t>(pos % kPage);
      };
      int32_t next = find(0);
      for (int j = 0; ok && j < walk.count; ++j) {
        const int32_t slot = next;
        const int k = tiles + j;
        const int ld = loads + (team == 0 ? pos_k(j) : pos_v(j, walk.count));
        const int sk = ld % C::kStages;
        constexpr int kLanes = F8 ? D / 16 : D / 8;    // lanes per key, 16 bytes each
        constexpr int kKeys = 32 / kLanes;             // keys per step of the warp
        uint4 v[kLanes];
        const int64_t off = slot < 0 ? -1
                                     : (static_cast<int64_t>(slot / kPage) * p.cache.page_stride +
                                        (slot % kPage) * p.cache.token_stride + walk.head * p.cache.head_stride) *
                                           (F8 ? 1 : 2);
#pragma unroll
        for (int x = 0; x < kLanes; ++x) {
          const int64_t o = __shfl_sync(0xffffffffu, off, x * kKeys + lane / kLanes);
          v[x] = o < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4 *>(cache + o) + lane % kLanes);
        }
        float sc = 0.0f;
        if (F8 && slot >= 0) sc = scales[(static_cast<int64_t>(slot / kPage) * Hkv + walk.head) * kPage + slot % kPage];
        if (j + 1 < walk.count) next = find(j + 1);
        const uint32_t bits = __ballot_sync(0xffffffffu, slot >= 0);
        if (!warp_wait_all(&bars.kv_empty[sk], ((ld / C::kStages) & 1) ^ 1) ||
            (F8 && !warp_wait_all(&bars.sc_empty[k % 8], ((k / 8) & 1) ^ 1))) {
          ok = false;
          break;
        }
        uint8_t *const dst = skv + sk * C::kTileBytes;
#pragma unroll
        for (int x = 0; x < kLanes; ++x) {
          const int key = w4 * 32 + x * kKeys + lane / kLanes, ch = lane % kLanes;
          if (F8) {
            uint8_t *const row = dst + (ch >> 2) * kBlockBytes + key * 128;
            const int c0 = (ch & 3) * 2;
            const uint2 a0 = e4m3x4_to_bf16(v[x].x), a1 = e4m3x4_to_bf16(v[x].y), a2 = e4m3x4_to_bf16(v[x].z),
                        a3 = e4m3x4_to_bf16(v[x].w);
            *reinterpret_cast<uint4 *>(row + ((c0 ^ (key & 7)) << 4)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
            *reinterpret_cast<uint4 *>(row + (((c0 + 1) ^ (key & 7)) << 4)) = make_uint4(a2.x, a2.y, a3.x, a3.y);
          } else {
            uint8_t *const row = dst + (ch >> 3) * kBlockBytes + key * 128;
            *reinterpret_cast<uint4 *>(row + (((ch & 7) ^ (key & 7)) << 4)) = v[x];
          }
        }
        if (F8) {
          ssc[(k % 8) * 2 * kTile + team * kTile + t] = sc;
          mbar_arrive(&bars.sc_full[k % 8]);
        }
        if (team == 0 && lane == 0) bars.keys_ok[k & 15][w4] = bits;
        fence_proxy_async_shared();
        mbar_arrive(&bars.kv_full[sk]);
      }
      loads += 2 * walk.count;
      tiles += walk.count;
    }
    if (!ok) give_up();
  }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------- combine
// Joins the shares of split items: one warp per (row, query head), lanes across the
// dimensions, the shares in CTA order.
template <int D, bool PAIR, bool SEL>
__global__ void __launch_bounds__(256) combine_kernel(const TreeAttnArgs a, int ctas) {
  constexpr int E = D / 32;
  constexpr int kSlotRows = PAIR ? 2 * kRows : kRows;
  const idx_tree_problem &p = a.p;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(p.R) * p.Hq) return;
  const int r = static_cast<int>(w / p.Hq), hq = static_cast<int>(w % p.Hq);
  int i = -1;   // the row's request: the last one that starts at or before it
  for (int i0 = 0; i0 < p.Q; i0 += 32) {
    const bool at = i0 + lane < p.Q && p.row_start[i0 + lane] <= r;
    i += __popc(__ballot_sync(0xffffffffu, at));
  }
  grid_dependency_wait();
  if (i < 0) return;
  const Req q = load_req<SEL>(a, i);
  const int t = r - q.row0;
  if (t < 0 || t >= q.tokens) return;
  const int64_t W = a.prefix[p.Q];
  const int G = p.Hq / p.cache.Hkv;
  const int head = hq / G, block = t / a.item_tokens;
  const int64_t b = a.prefix[i] + (static_cast<int64_t>(head) * q.blocks + block) * q.tiles, e = b + q.tiles;
  const int n = share_count(W, ctas);
  // the CTAs of the item's first and last tile
  auto owner = [&](int64_t x) {
    int c = static_cast<int>(min(static_cast<int64_t>(n - 1), x * n / W));
    while (share_begin(W, n, c) > x) --c;
    while (c + 1 < n && share_begin(W, n, c + 1) <= x) ++c;
    return c;
  };
  const int c0 = owner(b), c1 = owner(e - 1);
  if (c0 == c1) return;   // written whole
  const int tb = PAIR ? a.item_tokens / 2 : a.item_tokens;
  const int u = t - block * a.item_tokens;
  const int prow = (PAIR && u >= tb ? kRows + (u - tb) * G : u * G) + hq % G;
  // CTA c's share of the item is its first segment (slot 0) unless the item begins inside it
  auto slot_of = [&](int c) { return 2 * c + (share_begin(W, n, c) < b ? 1 : 0); };
  float m = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32)
    m = fmaxf(m, a.part_ml[static_cast<int64_t>(slot_of(c)) * kSlotRows + prow].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.0f, acc[E];
#pragma unroll
  for (int x = 0; x < E; ++x) acc[x] = 0.0f;
  for (int cb = c0; cb <= c1; cb += 32) {
    float f = 0.0f, lc = 0.0f;
    if (cb + lane <= c1) {
      const float2 ml = a.part_ml[static_cast<int64_t>(slot_of(cb + lane)) * kSlotRows + prow];
      f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
      lc = ml.y;
    }
    const int nc = min(32, c1 - cb + 1);
#pragma unroll 8
    for (int x = 0; x < nc; ++x) {
      const float fx = __shfl_sync(0xffffffffu, f, x), lx = __shfl_sync(0xffffffffu, lc, x);
      const float *const o = a.part_o + (static_cast<int64_t>(slot_of(cb + x)) * kSlotRows + prow) * D + lane * E;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(o);
        if (fx != 0.0f) {
          l += fx * lx;
          acc[0] += fx * v.x;
          acc[1] += fx * v.y;
          acc[2] += fx * v.z;
          acc[3] += fx * v.w;
        }
      } else {
        const float2 v = *reinterpret_cast<const float2 *>(o);
        if (fx != 0.0f) {
          l += fx * lx;
          acc[0] += fx * v.x;
          acc[1] += fx * v.y;
        }
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t *const out = a.out + (static_cast<int64_t>(r) * p.Hq + hq) * D + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t *>(out) = pack_bf16(acc[0] * inv, acc[1] * inv);
  if (lane == 0 && a.lse != nullptr)
    a.lse[static_cast<int64_t>(r) * p.Hq + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------------------- launch
template <int D, bool F8, bool PAIR, bool SEL>
cudaError_t launch(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm,
                   int num_sms, cudaStream_t stream) {
  using C = Cfg<D, F8, PAIR, SEL>;
  static std::mutex mu;
  static bool done[128] = {};
  const cudaError_t e = once_per_device(mu, done, [] {
    return cudaFuncSetAttribute(tree_attention_kernel<D, F8, PAIR, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::kDynamic);
  });
  if (e != cudaSuccess) return e;
  tree_attention_kernel<D, F8, PAIR, SEL><<<num_sms, C::kThreads, C::kDynamic, stream>>>(qm, km, vm, a);
  cudaError_t st = cudaGetLastError();
  if (st != cudaSuccess) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.p.R) * a.p.Hq + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<D, PAIR, SEL>, a, num_sms);
}

template <int D, bool F8>
cudaError_t launch_d(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm,
                     int num_sms, cudaStream_t stream) {
  if (a.sel != nullptr) return launch<D, F8, false, true>(a, qm, km, vm, num_sms, stream);
  if (a.pair) return launch<D, F8, true, false>(a, qm, km, vm, num_sms, stream);
  return launch<D, F8, false, false>(a, qm, km, vm, num_sms, stream);
}

}  // namespace

cudaError_t launch_tree_attention(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km,
                                  const CUtensorMap &vm, int num_sms, cudaStream_t stream) {
  const bool f8 = a.p.cache.kv_dtype == IDX_KV_E4M3;
  if (a.p.cache.D == 64)
    return f8 ? launch_d<64, true>(a, qm, km, vm, num_sms, stream) : launch_d<64, false>(a, qm, km, vm, num_sms, stream);
  return f8 ? launch_d<128, true>(a, qm, km, vm, num_sms, stream) : launch_d<128, false>(a, qm, km, vm, num_sms, stream);
}

}  // namespace idx
