// Attention of drafted tokens over a paged cache, whole or at selected positions.
//
// For a key/value head the query vectors that read it (tokens x query heads per
// key/value head) are the M = 128 rows of a tensor-core tile, and the 64 positions of
// a cache page its columns:
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
// Two streams fill the tensor core: the even and odd tiles of one row block (up to 128
// rows, joined in TMEM at the end of the item: more bytes in flight for the few-row,
// memory-bound calls) or two row blocks over the same tiles (more rows: each K and V
// tile is read from shared memory for 256 rows).  Each has O and two S buffers of 64
// columns in TMEM, so that the scores of a tile are computed while its four softmax
// warps, one thread per row, work on the tile before; P takes its S's place.
//
// A block of at most 32 (64) rows fills the 128 of the tile four (two) times over: Q
// is loaded that often, and each copy of the rows takes a quarter (half) of a tile's
// keys, with zeros in its P for the others.  All four softmax warps then work on
// every tile, 16 (32) keys each, and the copies' O are summed at the end of the item.
// The tensor core computes nothing that it would not have computed for the empty
// rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "idx_device.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr int kTile = kPage;             // keys per tile
constexpr int kRows = 128;               // rows of a stream
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // + 128 * stream (S: + 64 * buffer)
constexpr int kMinTiles = 4;             // tiles per CTA, at least (fewer CTAs otherwise)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's maximum moves only when a score passes it by 2^8: until then the sums run
// on the old one, below 2^8 * 2^19 in fp32, and O needs no pass through registers.
constexpr float kLazy = 8.0f;

// ---------------------------------------------------------------------------- roles
// warps 0-3 and 4-7: softmax of streams 0 and 1; 8: TMA producer; 9 and 10: MMA
// issuers of streams 0 and 1; 11: idle, or with 8 the gatherers of selected positions;
// 12-19 with an E4M3 cache: conversion to bf16, two teams of four on alternate loads.
constexpr int kProducerWarp = 8, kIssuerWarp = 9, kGatherWarp = 11, kConvertWarp = 12;

constexpr int kMaxStages = 16;

// COPIES: copies of the row block in the tile's rows (4, 2 or 1); PAIR: two row blocks.
template <int D, bool F8, int COPIES, bool PAIR, bool SEL>
struct Cfg {
  static constexpr int kTileBytes = kTile * D * 2;       // a K or V tile as bf16
  static constexpr int kRawBytes = kTile * D;            // ... as E4M3 bytes
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kQBufs = PAIR || F8 ? 1 : 2;
  static constexpr int kQTotal = kQBytes * (PAIR ? 2 : kQBufs);
  // bf16: 128 KB of tiles; E4M3: raw tiles as memory allows and 96 KB of converted ones
  static constexpr int kStages = F8 ? (D == 128 ? 6 : 12) : (D == 128 ? 8 : 16);
  static constexpr int kRawStages = !F8 ? 0 : D == 64 ? 16 : PAIR ? 6 : COPIES > 1 ? 8 : 10;
  static constexpr int kScaleStages = F8 ? 16 : 0;
  static constexpr int kRedBytes = COPIES > 1 ? 2 * kRows * 16 * 4 : 0;   // the copies' sum: 16 columns a stream
  static constexpr int kThreads = 32 * (F8 ? kConvertWarp + 8 : kConvertWarp);
  // K tiles loaded ahead of the first V: two per stream
  static constexpr int kAhead = PAIR ? 2 : 4;
  static_assert(kStages >= kAhead + 2 && kStages <= kMaxStages && kRawStages <= kMaxStages, "rings");
  // Registers per thread after the roles part, where a softmax thread holds up to 64
  // scores.  The shares add up to no more than the launch's threads x registers.
  static constexpr bool kShareRegs = F8;
  static constexpr int kRegsLaunch = 96, kRegsSoftmax = 144, kRegsOther = 64;
  static_assert(!F8 || 256 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * kRegsLaunch, "register shares");
  static constexpr int kDynamic = 1024 + kQTotal + kStages * kTileBytes + kRawStages * kRawBytes +
                                  kScaleStages * 2 * kTile * 4 + kRedBytes;
};

struct Barriers {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t raw_full[kMaxStages], raw_empty[kMaxStages];
  uint64_t sc_full[16], sc_empty[16];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2];   // [stream][buffer]
  uint64_t o_free[2], drain[2], stats[2], red_full[2], red_free[2], scrubbed[2];
  uint32_t tmem_base;
  int abort;
  int32_t two_terms[2][2];         // P of [stream][buffer] has a low term
  int32_t start_req, start_base;   // the share's first request, and the tiles before it
  uint32_t page_ok[32];            // dense: the page of the CTA's tile k % 32 was loaded
  uint32_t keys_ok[32][2];         // selected: bit per key of tile k % 32
  int32_t nonfinite[32];           // segment number + 1 whose drafted tokens' V held NaN or infinity
  float row_m[2][2][kRows], row_l[2][2][kRows];   // [segment parity][stream][row]
  int32_t warp_sums[20];
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
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
  q.keys = ctx + q.tokens;       // both far below 2^30
  const int64_t room = static_cast<int64_t>(p.pt_stride) * kPage;
  if (q.keys > room) {
    q.bad = kStatusBadBound;
    q.keys = static_cast<int32_t>(room);
  }
  const int n = a.sel != nullptr ? a.sel_k + q.tokens : q.keys;
  q.tiles = q.tokens > 0 ? (n + kTile - 1) / kTile : 0;
  q.blocks = (q.tokens + a.item_tokens - 1) / a.item_tokens;
  return q;
}
// Tiles of a request: with the host's bounds the launch's sum fits 31 bits.
__device__ __forceinline__ int req_tiles(const Req &q, int hkv) { return q.tiles * q.blocks * hkv; }

// Shares: W tiles over n CTAs, the first W % n of them with one more.
struct Shares {
  int W, n, per, rest;
  __device__ __forceinline__ Shares(int tiles, int ctas) : W(tiles) {
    n = max(1, min((tiles + kMinTiles - 1) / kMinTiles, ctas));
    per = W / n;
    rest = W - per * n;
  }
  __device__ __forceinline__ int begin(int c) const { return c * per + min(c, rest); }
  __device__ __forceinline__ int owner(int t) const {   // the CTA of tile t
    const int big = rest * (per + 1);
    return t < big ? t / (per + 1) : rest + (t - big) / per;
  }
};

// Walks the segments of a share: the tiles of one item that fall into it.
struct Walk {
  const TreeAttnArgs &a;
  int t, end, base;       // next tile, end of the share, tiles before request i
  int i;
  Req q;
  // the segment
  int seg = -1;           // its number
  int head, tok0, tokens; // key/value head; first token and token count of the item's block
  int tile0, count;       // first tile within the item, tiles
  bool whole;             // the segment is the whole item
  bool first;             // it is the share's first segment (its partial goes to slot 0)
  int share0;

  __device__ __forceinline__ Walk(const TreeAttnArgs &args, int t0, int t1, int req, int req_base)
      : a(args), t(t0), end(t1), base(req_base), i(req), share0(t0) {
    if (t < end) q = load_req(a, i);
  }
  __device__ __forceinline__ bool next() {
    if (t >= end) return false;
    int mine = req_tiles(q, a.p.cache.Hkv);
    while (t >= base + mine) {
      base += mine;
      q = load_req(a, ++i);
      mine = req_tiles(q, a.p.cache.Hkv);
    }
    const int off = t - base;
    const int item = off / q.tiles;
    tile0 = off - item * q.tiles;
    head = item / q.blocks;
    tok0 = (item - head * q.blocks) * a.item_tokens;
    tokens = min(a.item_tokens, q.tokens - tok0);
    count = min(end - t, q.tiles - tile0);
    whole = count == q.tiles;
    first = t == share0;
    t += count;
    ++seg;
    return true;
  }
};

// The loads of a segment of n tiles: K of the first `ahead` tiles, then V0, K, V1, K ...
// Their places in that order, and the load at place x.
__device__ __forceinline__ int pos_k(int j, int ahead) { return j < ahead ? j : 2 * j - ahead + 1; }
__device__ __forceinline__ int pos_v(int j, int n, int ahead) { return min(n, j + ahead) + j; }
__device__ __forceinline__ bool load_at(int x, int n, int ahead, int &j) {   // true: V of tile j, false: K
  const int lead = min(n, ahead);
  if (x < lead) {
    j = x;
    return false;
  }
  const int y = x - lead, both = 2 * (n - lead);
  if (y >= both) {
    j = n - lead + (y - both);
    return true;
  }
  j = (y >> 1) + (y & 1 ? lead : 0);
  return (y & 1) == 0;
}

// ---------------------------------------------------------------------------- softmax
// Moves the row's maximum to `top` where that passes it by more than kLazy, and scales l
// and O (D columns at to, once settled() says that the product before has completed)
// along; whole warps together.
template <int D, typename F>
__device__ __forceinline__ bool raise_maximum(uint32_t to, float top, bool has_o, float &m, float &l, F settled) {
  const bool grow = top > m + kLazy || (m == -INFINITY && top > -INFINITY);
  if (!__any_sync(0xffffffffu, grow)) return true;
  const float nm = fmaxf(m, top);
  const float f = m == -INFINITY ? 0.0f : ex2(m - nm);
  m = nm;
  l *= f;
  if (!has_o) return true;
  if (!settled()) return false;
#pragma unroll 1
  for (int w = 0; w < D / 16; ++w) {
    uint32_t x[16];
    tmem_ld16(to + 16 * w, x);
    tmem_wait_ld();
    reg_fence16(x);
#pragma unroll
    for (int y = 0; y < 16; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * f);
    tmem_st16(to + 16 * w, x);
  }
  return true;
}

// One row's keys of a tile (N of the 64, from column n0): S (columns at ts) to P in the
// same columns, the row's maximum m and sum l, and O (D columns at to) when the maximum
// moves.  special: only the keys of ok (a bit per key) are visible.  sc: the tile's K
// scales, then its V scales.
//
// P is rounded to bf16 for the product with V.  Over the 64 or more keys of a full tile
// the roundings average out below the output's own; the few keys of a special tile do
// not, so there P is kept in two bf16 terms, high in columns 0-31 and low in 32-63, and
// the product runs over both.
template <int D, bool F8, int N, typename F>
__device__ __forceinline__ bool softmax_tile(uint32_t ts, uint32_t to, const float *sc, float c, int n0, bool special,
                                             uint64_t ok, bool has_o, float &m, float &l, F settled) {
  constexpr int kW = N < 32 ? N : 32;        // columns per register group
  uint32_t x[N / kW][kW];
#pragma unroll
  for (int w = 0; w < N / kW; ++w) {
    if constexpr (kW == 32) tmem_ld32(ts + n0 + 32 * w, x[w]);
    else tmem_ld16(ts + n0, x[w]);
  }
  const float4 *const ks = reinterpret_cast<const float4 *>(sc + n0);
  const float2 *const vs = reinterpret_cast<const float2 *>(sc + kTile + n0);
  tmem_wait_ld();
#pragma unroll
  for (int w = 0; w < N / kW; ++w) {
    if constexpr (kW == 32) reg_fence32(x[w]);
    else reg_fence16(x[w]);
  }
  if (F8) {
#pragma unroll
    for (int w = 0; w < N / kW; ++w)
#pragma unroll
      for (int y = 0; y < kW; y += 4) {
        if (y % 16 == 0) asm volatile("" ::: "memory");   // at most four of the loads ahead
        const float4 k = ks[kW / 4 * w + y / 4];
        x[w][y] = __float_as_uint(__uint_as_float(x[w][y]) * k.x);
        x[w][y + 1] = __float_as_uint(__uint_as_float(x[w][y + 1]) * k.y);
        x[w][y + 2] = __float_as_uint(__uint_as_float(x[w][y + 2]) * k.z);
        x[w][y + 3] = __float_as_uint(__uint_as_float(x[w][y + 3]) * k.w);
      }
  }
  if (special) {
#pragma unroll
    for (int w = 0; w < N / kW; ++w)
#pragma unroll
      for (int y = 0; y < kW; ++y)
        x[w][y] = (static_cast<uint32_t>(ok >> (32 * w)) >> y) & 1u ? x[w][y] : 0xFF800000u;   // -infinity
  }
  float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int w = 0; w < N / kW; ++w)
#pragma unroll
    for (int y = 0; y < kW; y += 8)
#pragma unroll
      for (int z = 0; z < 4; ++z)
        t4[z] = max3(t4[z], __uint_as_float(x[w][y + 2 * z]), __uint_as_float(x[w][y + 2 * z + 1]));
  float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c;   // in units of log2
  if (top != top) top = 0.0f;   // scale 0: 0 x -inf moves no maximum
  if (!raise_maximum<D>(to, top, has_o, m, l, settled)) return false;
  const float base = m == -INFINITY ? 0.0f : m;
  const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
  float2 l2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int w = 0; w < N / kW; ++w) {
    uint32_t hi[kW / 2];
#pragma unroll
    for (int y = 0; y < kW; y += 2) {
      const float2 e2 = __ffma2_rn(make_float2(__uint_as_float(x[w][y]), __uint_as_float(x[w][y + 1])), c2, b2);
      float2 e = make_float2(ex2(e2.x), ex2(e2.y));
      l2[(y >> 1) & 1] = __fadd2_rn(l2[(y >> 1) & 1], e);
      if (F8) {
        if (y % 16 == 0) asm volatile("" ::: "memory");
        const float2 v = vs[kW / 2 * w + y / 2];
        if (special) {   // a stale scale may be NaN
          const uint32_t seen = static_cast<uint32_t>(ok >> (32 * w)) >> y;
          e.x = seen & 1u ? e.x * v.x : 0.0f;
          e.y = seen & 2u ? e.y * v.y : 0.0f;
        } else {
          e.x *= v.x;
          e.y *= v.y;
        }
      }
      hi[y / 2] = pack_bf16(e.x, e.y);
      x[w][y] = __float_as_uint(e.x);
      x[w][y + 1] = __float_as_uint(e.y);
    }
    if constexpr (kW == 32) tmem_st16(ts + n0 / 2 + 16 * w, hi);
    else tmem_st8(ts + n0 / 2, hi);
    if (special) {
      uint32_t lo[kW / 2];
#pragma unroll
      for (int y = 0; y < kW / 2; ++y) {
        // an infinity (a scale's) has no low term
        const float r0 = __uint_as_float(x[w][2 * y]) - __uint_as_float(hi[y] << 16);
        const float r1 = __uint_as_float(x[w][2 * y + 1]) - __uint_as_float(hi[y] & 0xFFFF0000u);
        lo[y] = pack_bf16(r0 == r0 ? r0 : 0.0f, r1 == r1 ? r1 : 0.0f);
      }
      if constexpr (kW == 32) tmem_st16(ts + 32 + n0 / 2 + 16 * w, lo);
      else tmem_st8(ts + 32 + n0 / 2, lo);
    }
  }
  if constexpr (N < kTile) {   // the other copies' keys
    uint32_t zero[8] = {};
#pragma unroll
    for (int w = 0; w < kTile / 2; w += 8) {
      if (w >= n0 / 2 && w < (n0 + N) / 2) continue;
      tmem_st8(ts + w, zero);
      if (special) tmem_st8(ts + 32 + w, zero);
    }
  }
  l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
  tmem_wait_st();
  return true;
}

// ---------------------------------------------------------------------------- kernel
template <int D, bool F8, int COPIES, bool PAIR, bool SEL>
__global__ void __launch_bounds__(Cfg<D, F8, COPIES, PAIR, SEL>::kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const TreeAttnArgs a) {
  using C = Cfg<D, F8, COPIES, PAIR, SEL>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Barriers bars;
  uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  uint8_t *const sq = smem;
  uint8_t *const skv = sq + C::kQTotal;
  uint8_t *const sraw = skv + C::kStages * C::kTileBytes;
  float *const ssc = reinterpret_cast<float *>(sraw + C::kRawStages * C::kRawBytes);   // [stage][K 64, V 64]
  float *const sred = ssc + C::kScaleStages * 2 * kTile;                                // [stream][row][16]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const idx_tree_problem &p = a.p;
  const int Hkv = p.cache.Hkv;
  const int G = p.Hq / Hkv;
  const int tb = PAIR ? a.item_tokens / 2 : a.item_tokens;   // tokens of a row block
  constexpr int kBlocks = D / 64;            // 64-dimension blocks of an operand tile
  constexpr int kBlockBytes = kTile * 128, kQBlockBytes = kRows * 128;
  grid_dependency_trigger();                 // the combine kernel's CTAs may take free SMs

  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      // filled by four converting warps, the two gathering ones or one TMA thread
      mbar_init(&bars.kv_full[s], F8 ? 4 : SEL ? 2 : 1);
      mbar_init(&bars.kv_empty[s], PAIR ? 2 : 1);
      mbar_init(&bars.raw_full[s], SEL ? 2 : 1);
      mbar_init(&bars.raw_empty[s], 4);
      mbar_init(&bars.sc_full[s], SEL ? 2 : 1);
      mbar_init(&bars.sc_empty[s], PAIR ? 8 : 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.q_full[s], 1);
      mbar_init(&bars.q_empty[s], 2);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars.s_full[s][b], 1);
        mbar_init(&bars.p_ready[s][b], 4);
        mbar_init(&bars.pv_done[s][b], 1);
      }
      mbar_init(&bars.o_free[s], PAIR ? 4 : 8);
      mbar_init(&bars.drain[s], 1);
      mbar_init(&bars.stats[s], 4);
      mbar_init(&bars.red_full[s], 4);
      mbar_init(&bars.red_free[s], 4);
      mbar_init(&bars.scrubbed[s], 4);
    }
    bars.abort = 0;
    for (int s = 0; s < 32; ++s) bars.nonfinite[s] = 0;
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
  // Every CTA sums the requests' tiles itself: a warp at a time for few requests, else
  // the whole CTA in chunks.
  constexpr int kWarps = C::kThreads / 32;
  int W = 0, req0 = 0, base0 = 0;
  uint32_t bad = 0;
  auto scan32 = [&](int i) -> int2 {   // (tiles of request i, inclusive sum over the warp)
    int mine = 0;
    if (i < p.Q) {
      const Req q = load_req(a, i);
      bad |= q.bad;
      mine = req_tiles(q, Hkv);
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    return make_int2(mine, incl);
  };
  if (p.Q <= 32) {
    const int2 s = scan32(lane);
    W = __shfl_sync(0xffffffffu, s.y, 31);
    const Shares sh(W, gridDim.x);
    const int t0 = sh.begin(min(static_cast<int>(blockIdx.x), sh.n));
    const uint32_t at = __ballot_sync(0xffffffffu, t0 >= s.y - s.x && t0 < s.y);
    if (at != 0u) {
      req0 = __ffs(at) - 1;
      base0 = __shfl_sync(0xffffffffu, s.y - s.x, req0);
    }
    if (blockIdx.x == 0 && warp == 0 && bad) flag_status(a.status, bad);
  } else {
    auto scan = [&](int i0, int before, int2 &s) -> int {   // sums of one chunk, returns its total
      s = scan32(i0 + tid);
      if (lane == 31) bars.warp_sums[warp] = s.y;
      __syncthreads();
      int total = 0;
      s.y += before;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) s.y += bars.warp_sums[w];
        total += bars.warp_sums[w];
      }
      __syncthreads();
      return total;
    };
    int2 s = make_int2(0, 0);
    for (int i0 = 0; i0 < p.Q; i0 += C::kThreads) W += scan(i0, W, s);
    if (blockIdx.x == 0 && bad) flag_status(a.status, bad);
    const Shares sh(W, gridDim.x);
    const int t0 = sh.begin(min(static_cast<int>(blockIdx.x), sh.n));
    int before = 0;
    for (int i0 = 0; i0 < p.Q; i0 += C::kThreads) {
      if (p.Q > C::kThreads) before += scan(i0, before, s);   // one chunk: the sums are still in registers
      if (i0 + tid < p.Q && t0 >= s.y - s.x && t0 < s.y) {
        bars.start_req = i0 + tid;
        bars.start_base = s.y - s.x;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const Shares share(W, gridDim.x);
  const bool idle = static_cast<int>(blockIdx.x) >= share.n || W == 0;
  const int t0 = idle ? 0 : share.begin(blockIdx.x), t1 = idle ? 0 : share.begin(blockIdx.x + 1);
  if (!idle && p.Q > 32) {
    req0 = bars.start_req;
    base0 = bars.start_base;
  }
  Walk walk(a, t0, t1, req0, base0);

  const uint64_t limit = a.wait_limit_ns;
  volatile int *abort = &bars.abort;
  int never = 0;
  // A wait whose outcome the whole warp shares (so that it leaves its loop together).
  auto warp_wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
    const bool r = mbar_wait(bar, parity, limit, abort);
    return __all_sync(0xffffffffu, r);
  };
  auto warp_arrive = [&](uint64_t *bar) {   // one arrival for the warp's threads
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto give_up = [&]() {
    flag_status(a.status, kStatusTimeout);
    *abort = 1;
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    if constexpr (C::kShareRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    constexpr int kBlockRows = kRows / COPIES;   // rows of a copy
    constexpr int kKeys = kTile / COPIES;        // keys of a tile that a copy takes
    const int s = warp >> 2;               // stream
    const int lrow = tid & 127;            // row of the stream's tile, and its TMEM lane
    const int row = lrow % kBlockRows;     // row of the block
    const int copy = lrow / kBlockRows;    // the same for a whole warp
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // first TMEM lane of the warp << 16
    const uint32_t to = tmem + kColO + 128 * s + lanes;
    const float c = p.scale * kLog2e;
    const int step = PAIR ? 1 : 2, j0 = PAIR ? 0 : s;
    int tiles = 0;      // tiles of earlier segments
    uint32_t n = 0;     // this stream's tiles so far
    uint32_t nred = 0;  // sums of copies so far
    bool ok = true;
    while (ok && walk.next()) {
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
        const int buf = n & 1;
        if ((F8 && !warp_wait_all(&bars.sc_full[k % 16], (k / 16) & 1)) ||
            !warp_wait_all(&bars.s_full[s][buf], (n >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint64_t okbits = ~0ull;   // the copy's keys of the tile that the row sees
        bool special;
        if (SEL) {
          const uint32_t k0 = bars.keys_ok[k & 31][0], k1 = bars.keys_ok[k & 31][1];
          special = (k0 & k1) != ~0u;
          if (special) okbits = (static_cast<uint64_t>(k1) << 32 | k0) >> (copy * kKeys);
        } else {
          const uint32_t page = bars.page_ok[k & 31];
          special = key0 + kTile > ctx || page == 0u;
          if (special) {
            const int lim = walk.q.keys - ctx;      // drafted tokens within the page table
            const uint64_t vm = lim >= 64 ? mask : mask & ((1ull << lim) - 1ull);
            const int before = ctx - key0;          // cached keys from the tile's first on
            if (before < 64) {
              if (before > 0) okbits = ((1ull << before) - 1ull) | (vm << before);
              else okbits = before > -64 ? vm >> -before : 0ull;
            }
            okbits = page != 0u ? okbits >> (copy * kKeys) : 0ull;
          }
        }
        if (!SEL && !F8 && special) {
          // V of tokens that some rows do not see has to be finite (0 x NaN is NaN): zero
          // what no row sees, and what is not finite among the drafted tokens (rows that
          // see it get it back at the end).  Two threads share a key.
          const int lv = 2 * tiles + pos_v(j, walk.count, C::kAhead);
          const int sv = lv % C::kStages;
          if (!warp_wait_all(&bars.kv_full[sv], (lv / C::kStages) & 1)) {
            ok = false;
            break;
          }
          const int key = lrow & 63, pos = key0 + key;
          const bool dead = pos >= walk.q.keys || bars.page_ok[k & 31] == 0u;
          if (dead || pos >= ctx) {
#pragma unroll 4
            for (int x = (lrow >> 6) * kBlocks * 4; x < (lrow >> 6) * kBlocks * 4 + kBlocks * 4; ++x) {
              uint4 *const at = reinterpret_cast<uint4 *>(skv + sv * C::kTileBytes + (x >> 3) * kBlockBytes + key * 128 +
                                                          ((x + key) & 7) * 16);
              uint4 v = dead ? make_uint4(0, 0, 0, 0) : *at;
              if (!dead) {
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
                bool changed = false;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  if ((w[y] & 0x7F80u) == 0x7F80u) {
                    w[y] &= 0xFFFF0000u;
                    changed = true;
                  }
                  if ((w[y] & 0x7F800000u) == 0x7F800000u) {
                    w[y] &= 0xFFFFu;
                    changed = true;
                  }
                }
                if (!changed) continue;
                bars.nonfinite[walk.seg & 31] = walk.seg + 1;
                v = make_uint4(w[0], w[1], w[2], w[3]);
              }
              *at = v;
            }
          }
          fence_proxy_async_shared();
          __syncwarp();
        }
        if (active) {
          // O may be touched once the product of the tile before has completed
          auto settled = [&]() { return warp_wait_all(&bars.pv_done[s][buf ^ 1], ((n - 1) >> 1) & 1); };
          if (!softmax_tile<D, F8, kKeys>(tmem + kColS + 128 * s + 64 * buf + lanes, to, ssc + (k % 16) * 2 * kTile, c,
                                          copy * kKeys, special, okbits, mine > 0, m, l, settled)) {
            ok = false;
            break;
          }
        }
        if (lrow == 0) bars.two_terms[s][buf] = special;
        tc_fence_before();
        warp_arrive(&bars.p_ready[s][buf]);
        if (F8 && lane == 0) mbar_arrive(&bars.sc_empty[k % 16]);
      }
      if (!ok) break;
      if (F8 && PAIR && !live)   // hand the scales of the tiles on
        for (int j = 0; j < walk.count; ++j) {
          const int k = tiles + j;
          if (!warp_wait_all(&bars.sc_full[k % 16], (k / 16) & 1)) {
            ok = false;
            break;
          }
          warp_arrive(&bars.sc_empty[k % 16]);
        }
      if (!ok) break;
      tiles += walk.count;

      // -------------------------------------------------------------- end of the segment
      // its last two products may still be under way
      if ((mine > 1 && !warp_wait_all(&bars.pv_done[s][n & 1], ((n - 2) >> 1) & 1)) ||
          (mine > 0 && !warp_wait_all(&bars.pv_done[s][(n - 1) & 1], ((n - 1) >> 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (l != l) m = INFINITY;   // a NaN among the visible scores takes the whole row, in every join
      float f0 = 1.0f, f1 = 0.0f;
      if (!PAIR) {
        // the row's maximum and sum over both streams and all copies; this thread's O
        // (of stream 0 and of stream 1) scales by f0 and f1
        const int sp = walk.seg & 1;
        bars.row_m[sp][s][lrow] = m;
        bars.row_l[sp][s][lrow] = l;
        tc_fence_before();
        warp_arrive(&bars.stats[s]);
        if (!warp_wait_all(&bars.stats[s], walk.seg & 1) || !warp_wait_all(&bars.stats[s ^ 1], walk.seg & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float mm = -INFINITY;
#pragma unroll
        for (int x = 0; x < 2 * COPIES; ++x) mm = fmaxf(mm, bars.row_m[sp][x & 1][(x >> 1) * kBlockRows + row]);
        l = 0.0f;
#pragma unroll
        for (int x = 0; x < 2 * COPIES; ++x) {
          const int at = (x >> 1) * kBlockRows + row;
          const float mx = bars.row_m[sp][x & 1][at];
          const float f = mx == -INFINITY ? 0.0f : ex2(mx - mm);
          l += bars.row_l[sp][x & 1][at] * f;
          if ((x >> 1) == copy) (x & 1 ? f1 : f0) = f;
        }
        m = mm;
      }
      const bool two = !PAIR && walk.count > 1;    // stream 1 has tiles
      const bool poison = *reinterpret_cast<volatile int32_t *>(&bars.nonfinite[walk.seg & 31]) == walk.seg + 1;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int hq = walk.head * G + row % G;
      const int slot = (walk.first ? 0 : 1) + 2 * static_cast<int>(blockIdx.x);
      const int prow = (PAIR ? s * kRows : 0) + row;
      constexpr int kSlotRows = PAIR ? 2 * kRows : kRows;
      // four columns of the row's output, from d on
      auto put = [&](int d, float4 o) {
        if (l == 0.0f) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (poison) {   // what was zeroed for the rows that do not see it
          float x[4] = {o.x, o.y, o.z, o.w};
          for (int u = 0; u < walk.q.tokens; ++u) {
            const int pos = ctx + u;
            if (!((mask >> u) & 1ull) || pos >= walk.q.keys || pos < walk.tile0 * kTile ||
                pos >= (walk.tile0 + walk.count) * kTile)
              continue;
            const int32_t pg = p.page_table[static_cast<int64_t>(walk.i) * p.pt_stride + pos / kPage];
            if (pg < 0 || pg >= p.cache.P) continue;
            const int64_t at = pg * p.cache.page_stride + (pos % kPage) * p.cache.token_stride +
                               walk.head * p.cache.head_stride + d;
            for (int y = 0; y < 4; ++y) {
              float v;
              if (F8) v = static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(p.cache.v)[at + y]);
              else v = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.cache.v)[at + y]);
              if (!isfinite(v)) x[y] += v;
            }
          }
          o = make_float4(x[0], x[1], x[2], x[3]);
        }
        if (walk.whole) {
          *reinterpret_cast<uint2 *>(a.out + (static_cast<int64_t>(r) * p.Hq + hq) * D + d) =
              make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        } else {
          *reinterpret_cast<float4 *>(a.part_o + (static_cast<int64_t>(slot) * kSlotRows + prow) * D + d) = o;
        }
      };
      if (row < nrow && copy == 0 && (PAIR || s == 0)) {
        if (!walk.whole) a.part_ml[static_cast<int64_t>(slot) * kSlotRows + prow] = make_float2(m, l);
        else if (a.lse != nullptr)
          a.lse[static_cast<int64_t>(r) * p.Hq + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      // O in chunks of 16 columns: both streams' half each, or one's all
      const uint32_t o0 = PAIR ? to : tmem + kColO + lanes;
#pragma unroll 1
      for (int d = PAIR ? 0 : s * (D / 2); d < (PAIR ? D : (s + 1) * (D / 2)); d += 16) {
        float o[16];
        if (active) {
          __syncwarp();
          uint32_t x[16], x1[16];
          tmem_ld16(o0 + d, x);
          if (two) tmem_ld16(o0 + 128 + d, x1);
          tmem_wait_ld();
          reg_fence16(x);
          reg_fence16(x1);
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            o[y] = PAIR ? __uint_as_float(x[y]) : f0 == 0.0f ? 0.0f : __uint_as_float(x[y]) * f0;
            if (two) o[y] += f1 == 0.0f ? 0.0f : __uint_as_float(x1[y]) * f1;
          }
        }
        if constexpr (COPIES == 1) {
          if (row < nrow)
#pragma unroll
            for (int y = 0; y < 16; y += 4) put(d + y, make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]));
        } else {
          // the copies' sum: thread (copy, row) takes 16 / COPIES of the columns
          float4 *const red = reinterpret_cast<float4 *>(sred) + s * kRows * 4;
          if (active)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              red[lrow * 4 + (y ^ ((lrow >> 1) & 3))] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          warp_arrive(&bars.red_full[s]);
          if (!warp_wait_all(&bars.red_full[s], nred & 1)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int z = 0; z < 4 / COPIES; ++z) {
            const int y = copy * (4 / COPIES) + z;
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (row < nrow) {
#pragma unroll
              for (int x = 0; x < COPIES; ++x) {
                const int at = x * kBlockRows + row;
                const float4 v = red[at * 4 + (y ^ ((at >> 1) & 3))];
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
              }
              put(d + 4 * y, sum);
            }
          }
          warp_arrive(&bars.red_free[s]);
          if (!warp_wait_all(&bars.red_free[s], nred & 1)) {
            ok = false;
            break;
          }
          ++nred;
        }
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.o_free[PAIR ? s : 0]);
        if (!PAIR) mbar_arrive(&bars.o_free[1]);
      }
    }
    if (!ok) give_up();
  } else if (warp < kConvertWarp) {
    if constexpr (C::kShareRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kProducerWarp || (SEL && warp == kGatherWarp)) {
      // -------------------------------------------------------------- producer
      int nload = 0;      // K and V tiles so far
      int nscale = 0;     // tiles with scales so far
      int nq = 0;         // Q loads so far
      bool ok = true;
      auto warp_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        int r = 1;
        if (lane == 0) r = mbar_wait(bar, parity, limit, abort);
        return __shfl_sync(0xffffffffu, r, 0) != 0;
      };
      // Gathering: copies of up to kPend tiles stay in flight while the next is issued;
      // their barriers are arrived on once the warp's copies have landed.
      constexpr int kPend = 4;
      uint64_t *pend[kPend] = {}, *pend_sc[kPend] = {};
      auto landed = [&](int x) {
        if (pend[x] == nullptr) return;
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          if (pend_sc[x] != nullptr) mbar_arrive(pend_sc[x]);
          mbar_arrive(pend[x]);
        }
        pend[x] = pend_sc[x] = nullptr;
      };
      auto flush = [&]() {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int x = 0; x < kPend; ++x) landed(x);
      };
      // A wait that never holds back copies that have landed: the wait's end may need them.
      auto wait_flushed = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (SEL && !__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) flush();
        return warp_wait(bar, parity);
      };
      while (ok && walk.next()) {
        // Q of the segment, once for every copy
        const int qb = walk.seg % C::kQBufs;
        if (warp == kProducerWarp) {
          if (!wait_flushed(&bars.q_empty[qb], ((walk.seg / C::kQBufs) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const int nhalf = PAIR && walk.tokens > tb ? 2 : 1;
            mbar_arrive_expect_tx(&bars.q_full[qb], static_cast<uint32_t>(nhalf * COPIES * kBlocks * G * tb * 128));
            for (int s = 0; s < nhalf; ++s)
              for (int b = 0; b < kBlocks; ++b)
                for (int x = 0; x < COPIES; ++x)
                  tma_load_3d(sq + (PAIR ? s : qb) * C::kQBytes + b * kQBlockBytes + x * (kQBlockBytes / COPIES), &qmap,
                              b * 64, walk.head * G, walk.q.row0 + walk.tok0 + s * tb, &bars.q_full[qb]);
          }
          ++nq;
        }
        if constexpr (SEL) {
          // ---------------------------------------------------------- gathering
          const int r = walk.q.row0 + walk.tok0;
          const uint64_t mask = p.mask != nullptr ? p.mask[r] : (2ull << walk.tok0) - 1ull;
          const int32_t *const sel = a.sel + static_cast<int64_t>(r) * a.sel_k;
          const int32_t *const table = p.page_table + static_cast<int64_t>(walk.i) * p.pt_stride;
          const int part = warp == kProducerWarp ? 0 : 32;   // the warp's keys of a tile: part + lane
          const int n0 = walk.tile0 * kTile + part + lane;
          // A key's way: its entry of the selection, its page, its slot; each step's load is
          // issued a tile or more ahead of the next step, so that none is waited for.
          auto entry = [&](int j) -> int32_t {
            const int n = n0 + j * kTile;
            return j < walk.count && n < a.sel_k ? sel[n] : -1;
          };
          auto position = [&](int j, int32_t e) -> int32_t {   // logical position, -1 for none
            const int n = n0 + j * kTile;
            if (j >= walk.count) return -1;
            if (n < a.sel_k) return e >= 0 && e < walk.q.ctx ? e : -1;
            const int u = n - a.sel_k;
            return u < walk.q.tokens && ((mask >> u) & 1ull) && walk.q.ctx + u < walk.q.keys ? walk.q.ctx + u : -1;
          };
          auto page_of = [&](int32_t pos) -> int32_t { return pos >= 0 ? table[pos / kPage] : -1; };
          auto slot_of = [&](int32_t pos, int32_t pg) -> int32_t {    // page * 64 + token, -1 for none
            if (pos < 0) return -1;
            if (pg < 0 || pg >= p.cache.P) {
              flag_status(a.status, kStatusBadPage);
              return -1;
            }
            return pg * kPage + pos % kPage;
          };
          int32_t e[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) e[x] = entry(x);
          int32_t pos[4], pg[4];   // tiles j .. j + 3
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            pos[x] = position(x, e[x]);
            pg[x] = page_of(pos[x]);
          }
          int32_t old[C::kAhead] = {};     // slots of tiles j - 1, j - 2 ..
          for (int j = 0; ok && j < walk.count + C::kAhead; ++j) {
            const int32_t cur = slot_of(pos[0], pg[0]);
            // V of tile j - kAhead, then K of tile j
            for (int what = 1; what >= 0; --what) {
              if (what == 0 ? j >= walk.count : j < C::kAhead) continue;
              constexpr int ring = F8 ? C::kRawStages : C::kStages;
              const int s = nload % ring;
              if (!wait_flushed(F8 ? &bars.raw_empty[s] : &bars.kv_empty[s], ((nload / ring) & 1) ^ 1)) {
                ok = false;
                break;
              }
              const int32_t slot = what == 0 ? cur : old[C::kAhead - 1];
              if (what == 0) {
                const uint32_t bits = __ballot_sync(0xffffffffu, slot >= 0);
                if (lane == 0) bars.keys_ok[nscale & 31][part / 32] = bits;
                if constexpr (F8) {
                  if (!wait_flushed(&bars.sc_empty[nscale % 16], ((nscale / 16) & 1) ^ 1)) {
                    ok = false;
                    break;
                  }
                  const int64_t at = slot < 0 ? 0
                                              : (static_cast<int64_t>(slot / kPage) * Hkv + walk.head) * kPage + slot % kPage;
                  float *const d = ssc + (nscale % 16) * 2 * kTile + part + lane;
#pragma unroll
                  for (int x = 0; x < 2; ++x)   // the key's K and V scales
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(d + x * kTile)),
                                 "l"((x == 0 ? p.cache.k_scale : p.cache.v_scale) + at), "r"(slot < 0 ? 0 : 4)
                                 : "memory");
                }
              }
              // 16 bytes per lane: D / 16 or D / 8 lanes bring one key
              constexpr int kLanes = F8 ? D / 16 : D / 8;
              constexpr int kKeysAtOnce = 32 / kLanes;
              const uint8_t *const cache = static_cast<const uint8_t *>(what == 0 ? p.cache.k : p.cache.v);
              uint8_t *const dst = F8 ? sraw + s * C::kRawBytes : skv + s * C::kTileBytes;
              const int ch = lane % kLanes;
              const int64_t off = slot < 0 ? -1
                                           : (static_cast<int64_t>(slot / kPage) * p.cache.page_stride +
                                              (slot % kPage) * p.cache.token_stride + walk.head * p.cache.head_stride) *
                                                 (F8 ? 1 : 2);
#pragma unroll 8
              for (int y = 0; y < kLanes; ++y) {
                const int from = y * kKeysAtOnce + lane / kLanes;
                const int64_t o = __shfl_sync(0xffffffffu, off, from);
                const int key = part + from;
                uint8_t *const at = F8 ? dst + key * D + ch * 16
                                       : dst + (ch >> 3) * kBlockBytes + key * 128 + (((ch & 7) ^ (key & 7)) << 4);
                const uint8_t *const src = cache + (o < 0 ? 0 : o) + ch * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(at)), "l"(src),
                             "r"(o < 0 ? 0 : 16)
                             : "memory");
              }
              asm volatile("cp.async.commit_group;" ::: "memory");
              asm volatile("cp.async.wait_group %0;" ::"n"(kPend) : "memory");
              landed(0);
#pragma unroll
              for (int x = 0; x + 1 < kPend; ++x) {
                pend[x] = pend[x + 1];
                pend_sc[x] = pend_sc[x + 1];
              }
              pend[kPend - 1] = F8 ? &bars.raw_full[s] : &bars.kv_full[s];
              pend_sc[kPend - 1] = F8 && what == 0 ? &bars.sc_full[nscale % 16] : nullptr;
              ++nload;
              if (what == 0) ++nscale;
            }
#pragma unroll
            for (int x = C::kAhead - 1; x > 0; --x) old[x] = old[x - 1];
            old[0] = cur;
#pragma unroll
            for (int x = 0; x < 3; ++x) {
              pos[x] = pos[x + 1];
              pg[x] = pg[x + 1];
            }
            pos[3] = position(j + 4, e[4]);
            pg[3] = page_of(pos[3]);
#pragma unroll
            for (int x = 4; x < 7; ++x) e[x] = e[x + 1];
            e[7] = entry(j + 8);
          }
        } else {
          // ---------------------------------------------------------- pages by TMA
          const int32_t *const table = p.page_table + static_cast<int64_t>(walk.i) * p.pt_stride + walk.tile0;
          // page ids of 32 tiles of the segment at a time (tiles are pages)
          auto fetch = [&](int j) -> int32_t { return j + lane < walk.count ? table[j + lane] : -1; };
          int32_t ids = fetch(0), ids_next = fetch(32), ids_old = -1;
          for (int j = 0; ok && j < walk.count + C::kAhead; ++j) {
            if (j > 0 && (j & 31) == 0) {
              ids_old = ids;
              ids = ids_next;
              ids_next = fetch(j + 32);
            }
            // V of tile j - kAhead, then K of tile j
            for (int what = 1; what >= 0; --what) {
              if (what == 0 ? j >= walk.count : j < C::kAhead) continue;
              const int tile = what == 0 ? j : j - C::kAhead;
              const int32_t pg = __shfl_sync(0xffffffffu, (tile >> 5) == (j >> 5) ? ids : ids_old, tile & 31);
              const bool good = pg >= 0 && pg < p.cache.P;
              constexpr int ring = F8 ? C::kRawStages : C::kStages;
              const int s = nload % ring;
              if (!warp_wait(F8 ? &bars.raw_empty[s] : &bars.kv_empty[s], ((nload / ring) & 1) ^ 1)) {
                ok = false;
                break;
              }
              uint8_t *const dst = F8 ? sraw + s * C::kRawBytes : skv + s * C::kTileBytes;
              uint64_t *const full = F8 ? &bars.raw_full[s] : &bars.kv_full[s];
              if (what == 0) {
                if (lane == 0) {
                  bars.page_ok[nscale & 31] = good;
                  if (!good) flag_status(a.status, kStatusBadPage);
                }
                if constexpr (F8) {
                  const int ss = nscale % 16;
                  if (!warp_wait(&bars.sc_empty[ss], ((nscale / 16) & 1) ^ 1)) {
                    ok = false;
                    break;
                  }
                  if (lane == 0) {
                    mbar_arrive_expect_tx(&bars.sc_full[ss], good ? 512u : 0u);
                    if (good) {
                      const int64_t at = (static_cast<int64_t>(pg) * Hkv + walk.head) * kPage;
                      bulk_load(ssc + ss * 2 * kTile, p.cache.k_scale + at, 256u, &bars.sc_full[ss]);
                      bulk_load(ssc + ss * 2 * kTile + kTile, p.cache.v_scale + at, 256u, &bars.sc_full[ss]);
                    }
                  }
                }
              }
              if (lane == 0) {
                const void *const map = what == 0 ? &kmap : &vmap;
                mbar_arrive_expect_tx(full, good ? static_cast<uint32_t>(F8 ? C::kRawBytes : C::kTileBytes) : 0u);
                if (good) {
                  if constexpr (F8) {
                    tma_load_4d(dst, map, 0, 0, walk.head, pg, full);
                  } else {
                    for (int b = 0; b < kBlocks; ++b)
                      tma_load_4d(dst + b * kBlockBytes, map, b * 64, 0, walk.head, pg, full);
                  }
                }
              }
              ++nload;
              if (what == 0) ++nscale;
            }
          }
        }
      }
      if (SEL) flush();
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
        if (warp == kProducerWarp) land(bars.q_full, C::kQBufs, nq);
        if (!SEL) {
          if constexpr (F8) land(bars.raw_full, C::kRawStages, nload);
          else land(bars.kv_full, C::kStages, nload);
          if (F8) land(bars.sc_full, 16, nscale);
        }
      }
    } else if (warp == kIssuerWarp || warp == kIssuerWarp + 1) {
      // -------------------------------------------------------------- MMA issuers
      // Per stream: S of two tiles; then, tile by tile, O += P V once its P is ready, and S
      // of the second next tile once that has completed, since it takes P's columns.
      if (lane == 0) {
        const int s = warp - kIssuerWarp;
        const uint32_t ts = tmem + kColS + 128 * s, to = tmem + kColO + 128 * s;
        const uint32_t idesc_s = umma_idesc(1u, kTile), idesc_o = umma_idesc(1u, D) | kIdescBMn;
        int loads = 0;      // K and V tiles of earlier segments
        uint32_t ns = 0;    // this stream's S so far
        uint32_t n = 0;     // this stream's products with V so far
        bool ok = true, any = false;
        while (ok && walk.next()) {
          const int qb = walk.seg % C::kQBufs;
          const bool live = !PAIR || s == 0 || walk.tokens > tb;   // this stream has rows
          if (!mbar_wait(&bars.q_full[qb], (walk.seg / C::kQBufs) & 1, limit, abort)) {
            ok = false;
            break;
          }
          const uint64_t qdesc = umma_desc_sw128(smem_u32(sq + (PAIR ? s : qb) * C::kQBytes));
          const int step = PAIR ? 1 : 2, j0 = PAIR ? 0 : s;
          if (j0 >= walk.count) mbar_arrive(&bars.q_empty[qb]);
          auto scores = [&](int j) -> bool {   // S of tile j
            const int lk = loads + pos_k(j, C::kAhead);
            const int sk = lk % C::kStages;
            if (!mbar_wait(&bars.kv_full[sk], (lk / C::kStages) & 1, limit, abort)) return false;
            const bool last = j + step >= walk.count;
            if (!live) {   // no rows: only pass the tile on
              mbar_arrive(&bars.kv_empty[sk]);
              if (last) mbar_arrive(&bars.q_empty[qb]);
              return true;
            }
            tc_fence_after();
            const uint64_t kdesc = umma_desc_sw128(smem_u32(skv + sk * C::kTileBytes));
            const uint32_t d = ts + 64 * (ns & 1);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_f16(d, qdesc + (((kk >> 2) * kQBlockBytes + (kk & 3) * 32) >> 4),
                       kdesc + (((kk >> 2) * kBlockBytes + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
            umma_commit(&bars.s_full[s][ns & 1]);
            umma_commit(&bars.kv_empty[sk]);
            if (last) umma_commit(&bars.q_empty[qb]);
            any = true;
            ++ns;
            return true;
          };
          for (int j = j0; ok && j < walk.count && j < j0 + 2 * step; j += step) ok = scores(j);
          for (int j = j0; ok && j < walk.count; j += step) {
            const int lv = loads + pos_v(j, walk.count, C::kAhead);
            const int sv = lv % C::kStages, buf = n & 1;
            if (!live) {
              ok = mbar_wait(&bars.kv_full[sv], (lv / C::kStages) & 1, limit, abort);
              if (!ok) break;
              mbar_arrive(&bars.kv_empty[sv]);
            } else {
              if (!mbar_wait(&bars.p_ready[s][buf], (n >> 1) & 1, limit, abort) ||
                  (j == j0 && !mbar_wait(&bars.o_free[s], (walk.seg & 1) ^ 1, limit, abort)) ||
                  !mbar_wait(&bars.kv_full[sv], (lv / C::kStages) & 1, limit, abort)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t vdesc = umma_desc_mn(smem_u32(skv + sv * C::kTileBytes), kBlockBytes);
              const uint32_t ta = ts + 64 * buf;
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                umma_f16_ta(to, ta + kk * 8, vdesc + ((kk * 2048) >> 4), idesc_o, j > j0 || kk > 0);
              if (*reinterpret_cast<volatile int32_t *>(&bars.two_terms[s][buf])) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                  umma_f16_ta(to, ta + 32 + kk * 8, vdesc + ((kk * 2048) >> 4), idesc_o, 1u);
              }
              umma_commit(&bars.pv_done[s][buf]);
              umma_commit(&bars.kv_empty[sv]);
              ok = mbar_wait(&bars.pv_done[s][buf], (n >> 1) & 1, limit, abort);
              if (!ok) break;
              ++n;
            }
            if (j + 2 * step < walk.count) ok = scores(j + 2 * step);
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
    }
  } else {
    if constexpr (F8) {
      // -------------------------------------------------------------- E4M3 to bf16
      if constexpr (C::kShareRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
      const int team = (warp - kConvertWarp) >> 2, t = (tid - kConvertWarp * 32) & 127;
      int loads = 0, tiles = 0;     // of earlier segments
      uint32_t scrubs = 0;
      bool ok = true;
      while (ok && walk.next()) {
        for (int x = (loads ^ team) & 1; ok && x < 2 * walk.count; x += 2) {   // the team's loads: every second one
          int j;
          const bool is_v = load_at(x, walk.count, C::kAhead, j);
          const int load = loads + x;
          const int sr = load % C::kRawStages, sk = load % C::kStages;
          if (!warp_wait_all(&bars.raw_full[sr], (load / C::kRawStages) & 1)) {
            ok = false;
            break;
          }
          uint8_t *const src = sraw + sr * C::kRawBytes;
          uint8_t *const dst = skv + sk * C::kTileBytes;
          if (!SEL && is_v) {
            const int key0 = (walk.tile0 + j) * kTile;
            const bool page = bars.page_ok[(tiles + j) & 31] != 0u;
            if (key0 + kTile > walk.q.ctx || !page) {
              // V of tokens that some rows do not see has to be finite (0 x NaN is NaN): zero
              // what no row sees, and the NaN codes among the drafted tokens (rows that see
              // them get them back at the end).  Two threads share a key.
              const int key = t & 63, pos = key0 + key;
              const bool dead = pos >= walk.q.keys || !page;
              if (dead || pos >= walk.q.ctx) {
#pragma unroll 4
                for (int y = 0; y < D / 8; ++y) {
                  uint32_t *const at = reinterpret_cast<uint32_t *>(src + key * D) + (t >> 6) * (D / 8) + (y + t) % (D / 8);
                  uint32_t w = dead ? 0u : *at;
#pragma unroll
                  for (int z = 0; z < 32; z += 8)
                    if (((w >> z) & 0x7Fu) == 0x7Fu) {
                      w &= ~(0xFFu << z);
                      bars.nonfinite[walk.seg & 31] = walk.seg + 1;
                    }
                  *at = w;
                }
              }
              warp_arrive(&bars.scrubbed[team]);
              if (!warp_wait_all(&bars.scrubbed[team], scrubs & 1)) {
                ok = false;
                break;
              }
              ++scrubs;
            }
          }
          constexpr int kChunks = D / 16;             // 16-byte chunks of codes per key
          constexpr int kBatch = kTile * kChunks / 128;   // chunks per thread
          uint4 v[kBatch];
#pragma unroll
          for (int y = 0; y < kBatch; ++y) v[y] = *reinterpret_cast<const uint4 *>(src + (y * 128 + t) * 16);
          if (!warp_wait_all(&bars.kv_empty[sk], ((load / C::kStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int y = 0; y < kBatch; ++y) {
            const int key = (y * 128 + t) / kChunks, ch = t % kChunks;
            const uint2 a0 = e4m3x4_to_bf16(v[y].x), a1 = e4m3x4_to_bf16(v[y].y), a2 = e4m3x4_to_bf16(v[y].z),
                        a3 = e4m3x4_to_bf16(v[y].w);
            uint8_t *const row = dst + (ch >> 2) * kBlockBytes + key * 128;
            const int c0 = (ch & 3) * 2;
            *reinterpret_cast<uint4 *>(row + ((c0 ^ (key & 7)) << 4)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
            *reinterpret_cast<uint4 *>(row + (((c0 + 1) ^ (key & 7)) << 4)) = make_uint4(a2.x, a2.y, a3.x, a3.y);
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars.kv_full[sk]);
            mbar_arrive(&bars.raw_empty[sr]);
          }
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
// dimensions, the shares in CTA order.  All that depends on the inputs alone is worked
// out while the attention kernel still runs.
template <int D>
__global__ void __launch_bounds__(256) combine_kernel(const TreeAttnArgs a, int ctas) {
  constexpr int E = D / 32;
  const idx_tree_problem &p = a.p;
  const int slot_rows = a.pair ? 2 * kRows : kRows;
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= p.R * p.Hq) return;
  const int r = w / p.Hq, hq = w - r * p.Hq;
  const int Hkv = p.cache.Hkv;
  int i = -1, W = 0, upto = 0;   // the row's request: the last one that starts at or before it
  for (int i0 = 0; i0 < p.Q; i0 += 32) {
    int tiles = 0;
    bool at = false;
    if (i0 + lane < p.Q) {
      tiles = req_tiles(load_req(a, i0 + lane), Hkv);
      at = p.row_start[i0 + lane] <= r;
    }
    i += __popc(__ballot_sync(0xffffffffu, at));
    W += __reduce_add_sync(0xffffffffu, tiles);
    upto += __reduce_add_sync(0xffffffffu, at ? tiles : 0);
  }
  if (i < 0 || W == 0) return;
  const Req q = load_req(a, i);
  const int t = r - q.row0;
  if (t < 0 || t >= q.tokens) return;
  const int G = p.Hq / Hkv;
  const int head = hq / G, block = t / a.item_tokens;
  const int b = upto - req_tiles(q, Hkv) + (head * q.blocks + block) * q.tiles, e = b + q.tiles;
  const Shares sh(W, ctas);
  const int c0 = sh.owner(b), c1 = sh.owner(e - 1);
  if (c0 == c1) return;   // written whole
  const int tb = a.pair ? a.item_tokens / 2 : a.item_tokens;
  const int u = t - block * a.item_tokens;
  const int prow = (u >= tb ? kRows + (u - tb) * G : u * G) + hq - head * G;
  // CTA c's share of the item is its first segment (slot 0) unless the item begins inside it
  const int slot0 = 2 * c0 + (sh.begin(c0) < b ? 1 : 0);
  auto slot_of = [&](int c) { return c == c0 ? slot0 : 2 * c; };
  grid_dependency_wait();
  float m = -INFINITY, l = 0.0f, acc[E];
#pragma unroll
  for (int x = 0; x < E; ++x) acc[x] = 0.0f;
  for (int cb = c0; cb <= c1; cb += 32) {
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (cb + lane <= c1) ml = a.part_ml[static_cast<int64_t>(slot_of(cb + lane)) * slot_rows + prow];
    // the maximum so far, and what was summed up on the old one
    float nm = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, o));
    nm = fmaxf(nm, m);
    const float keep = m == -INFINITY ? 0.0f : ex2(m - nm);
    m = nm;
    l *= keep;
#pragma unroll
    for (int x = 0; x < E; ++x) acc[x] *= keep;
    const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - nm);
    const int nc = min(32, c1 - cb + 1);
#pragma unroll 8
    for (int x = 0; x < nc; ++x) {
      const float fx = __shfl_sync(0xffffffffu, f, x), lx = __shfl_sync(0xffffffffu, ml.y, x);
      const float *const o = a.part_o + (static_cast<int64_t>(slot_of(cb + x)) * slot_rows + prow) * D + lane * E;
      float v[E];
      if constexpr (E == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(o);
      else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(o);
      if (fx != 0.0f) {
        l += fx * lx;
#pragma unroll
        for (int y = 0; y < E; ++y) acc[y] += fx * v[y];
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
template <int D, bool F8, int COPIES, bool PAIR, bool SEL>
cudaError_t launch(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm,
                   int num_ctas, cudaStream_t stream) {
  using C = Cfg<D, F8, COPIES, PAIR, SEL>;
  static std::mutex mu;
  static bool done[128] = {};
  const cudaError_t e = once_per_device(mu, done, [] {
    if (C::kShareRegs) {
      // the register shares come out of what the launch gets: a smaller launch would wait forever
      cudaFuncAttributes f;
      const cudaError_t got = cudaFuncGetAttributes(&f, tree_attention_kernel<D, F8, COPIES, PAIR, SEL>);
      if (got != cudaSuccess) return got;
      if (f.numRegs != C::kRegsLaunch) return cudaErrorInvalidConfiguration;
    }
    return cudaFuncSetAttribute(tree_attention_kernel<D, F8, COPIES, PAIR, SEL>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kDynamic);
  });
  if (e != cudaSuccess) return e;
  tree_attention_kernel<D, F8, COPIES, PAIR, SEL><<<num_ctas, C::kThreads, C::kDynamic, stream>>>(qm, km, vm, a);
  cudaError_t st = cudaGetLastError();
  if (st != cudaSuccess) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.p.R * a.p.Hq + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<D>, a, num_ctas);
}

template <int D, bool F8, bool SEL>
cudaError_t launch_shape(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm,
                         int num_ctas, cudaStream_t stream) {
  if constexpr (!SEL)
    if (a.pair) return launch<D, F8, 1, true, SEL>(a, qm, km, vm, num_ctas, stream);
  if (a.copies == 4) return launch<D, F8, 4, false, SEL>(a, qm, km, vm, num_ctas, stream);
  if (a.copies == 2) return launch<D, F8, 2, false, SEL>(a, qm, km, vm, num_ctas, stream);
  return launch<D, F8, 1, false, SEL>(a, qm, km, vm, num_ctas, stream);
}

}  // namespace
}  // namespace idx
