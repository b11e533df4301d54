// What the attention kernels share: tensor-memory and tensor-map helpers, the plan that
// deals a launch's tiles out to the CTAs, and the join of split items.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "idx_device.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's probabilities are powers of two relative to a reference that moves only when a
// score passes it by 2^30: bf16 and fp32 hold what lies above (sums stay below 2^30 x 2^19)
// as exactly as what lies below, and O seldom needs a pass through registers.
constexpr float kLazy = 30.0f;

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
// Descriptor of a K-major operand with rows of 64 bytes in the 64-byte swizzle.
__device__ __forceinline__ uint64_t umma_desc_sw64(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(512u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(4u) << 61;
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
// Two floats to their nearest E4M3 codes (low byte: a).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t x) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x), __NV_E4M3)));
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
  q.keys = ctx + q.tokens;       // at most 2^30 + 64
  const int64_t room = static_cast<int64_t>(p.pt_stride) * kPage;
  if (q.keys > room) {
    q.bad = kStatusBadBound;
    q.keys = static_cast<int32_t>(room);
  }
  const int n = a.sel != nullptr ? a.sel_k + q.tokens : q.keys;
  q.tiles = q.tokens > 0 ? (n + a.tile - 1) / a.tile : 0;
  q.blocks = (q.tokens + a.item_tokens - 1) / a.item_tokens;
  return q;
}
// Tiles of a request.  With the host's bounds the launch's sum is below INT32_MAX, unless
// requests share rows (row_start does not ascend): sums stop there, and such a launch does nothing.
__device__ __forceinline__ int req_tiles(const Req &q, int hkv) { return q.tiles * q.blocks * hkv; }
__device__ __forceinline__ int add_tiles(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), static_cast<uint32_t>(INT32_MAX)));
}

constexpr int kMinKeys = 256;   // keys of a CTA's share, at least (fewer CTAs otherwise)

// Shares: W tiles over n CTAs, the first W % n of them with one more.
struct Shares {
  int W, n, per, rest;
  __device__ __forceinline__ Shares(int tiles, int tile, int ctas) : W(tiles) {
    const int least = tiles <= ctas ? 1 : kMinKeys / tile;
    n = max(1, min((tiles + least - 1) / least, ctas));
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

  __device__ __forceinline__ Walk(const TreeAttnArgs &args, int t0, int t1, int req, int req_base, const Req &first)
      : a(args), t(t0), end(t1), base(req_base), i(req), q(first), share0(t0) {}
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

// The CTA's share of the launch's tiles: every CTA sums the requests' tiles itself, a warp
// at a time for few requests, else the whole CTA in chunks.  Whole CTAs call it; with more
// than 32 requests `found` holds the share's first request after the next __syncthreads.
struct Start {
  int W;            // tiles of the launch
  int req, base;    // the share's first request, and the tiles before it
  Req q;            // that request
};
template <int kThreads>
__device__ __forceinline__ Start find_share(const TreeAttnArgs &a, Start *found, int *warp_sums) {
  const idx_tree_problem &p = a.p;
  const int Hkv = p.cache.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kThreads / 32;
  Start st{};
  Req q{};
  uint32_t bad = 0;
  auto scan32 = [&](int i) -> int2 {   // (tiles of request i, inclusive sum over the warp)
    int mine = 0;
    if (i < p.Q) {
      q = load_req(a, i);
      bad |= q.bad;
      mine = req_tiles(q, Hkv);
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = add_tiles(incl, up);
    }
    return make_int2(mine, incl);
  };
  if (p.Q <= 32) {
    const int2 s = scan32(lane);
    st.W = __shfl_sync(0xffffffffu, s.y, 31);
    if (st.W == INT32_MAX) {
      st.W = 0;
      bad |= kStatusBadBound;
    }
    const Shares sh(st.W, a.tile, gridDim.x);
    const int t0 = sh.begin(min(static_cast<int>(blockIdx.x), sh.n));
    const uint32_t at = __ballot_sync(0xffffffffu, t0 >= s.y - s.x && t0 < s.y);
    st.req = at != 0u ? __ffs(at) - 1 : 0;
    st.base = __shfl_sync(0xffffffffu, s.y - s.x, st.req);
    st.q.row0 = __shfl_sync(0xffffffffu, q.row0, st.req);
    st.q.tokens = __shfl_sync(0xffffffffu, q.tokens, st.req);
    st.q.ctx = __shfl_sync(0xffffffffu, q.ctx, st.req);
    st.q.keys = __shfl_sync(0xffffffffu, q.keys, st.req);
    st.q.tiles = __shfl_sync(0xffffffffu, q.tiles, st.req);
    st.q.blocks = __shfl_sync(0xffffffffu, q.blocks, st.req);
    if (blockIdx.x == 0 && warp == 0 && bad) flag_status(a.status, bad);
    return st;
  }
  auto scan = [&](int i0, int before, int2 &s) -> int {   // sums of one chunk, returns its total
    s = scan32(i0 + tid);
    if (lane == 31) warp_sums[warp] = s.y;
    __syncthreads();
    int total = 0;
    s.y = add_tiles(s.y, before);
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) s.y = add_tiles(s.y, warp_sums[w]);
      total = add_tiles(total, warp_sums[w]);
    }
    __syncthreads();
    return total;
  };
  int2 s = make_int2(0, 0);
  for (int i0 = 0; i0 < p.Q; i0 += kThreads) st.W = add_tiles(st.W, scan(i0, st.W, s));
  if (st.W == INT32_MAX) {
    if (blockIdx.x == 0 && tid == 0) flag_status(a.status, kStatusBadBound);
    st.W = 0;
    return st;
  }
  if (blockIdx.x == 0 && bad) flag_status(a.status, bad);
  const Shares sh(st.W, a.tile, gridDim.x);
  const int t0 = sh.begin(min(static_cast<int>(blockIdx.x), sh.n));
  int before = 0;
  for (int i0 = 0; i0 < p.Q; i0 += kThreads) {
    if (p.Q > kThreads) before = add_tiles(before, scan(i0, before, s));   // one chunk: the sums are still in registers
    if (i0 + tid < p.Q && t0 >= s.y - s.x && t0 < s.y) {
      found->req = i0 + tid;
      found->base = s.y - s.x;
      found->q = q;
    }
  }
  return st;
}

// ---------------------------------------------------------------------------- join
// A split item is joined by the CTAs that share it.  Each leaves its share (O before the
// division, the rows' references and sums) in its slot of the state and counts itself in;
// once all are in, each joins its part of the item's outputs, four values at a time, in CTA
// order.  The launch is cooperative: the CTAs that wait for each other run at the same time.
struct Share {
  int row0, head, nrow;   // the item's first row of q, key/value head, rows
  int c0, count;          // its first CTA, and how many there are
  int slot0;              // the first CTA's slot (the others': 2 * CTA)
};

// The segment's part in a join; begin: the item's first tile in the launch's order.
__device__ __forceinline__ Share share_of(const Walk &w, const Shares &sh, int G) {
  Share s;
  const int begin = w.t - w.count - w.tile0;
  s.row0 = w.q.row0 + w.tok0;
  s.head = w.head;
  s.nrow = w.tokens * G;
  s.c0 = sh.owner(begin);
  s.count = sh.owner(begin + w.q.tiles - 1) - s.c0 + 1;
  s.slot0 = 2 * s.c0 + (sh.begin(s.c0) < begin ? 1 : 0);
  return s;
}

// A share's O: rows of D values, as the few-row kernel's threads (one per dimension) hold
// them, or (BY_FOURS) groups of four dimensions of all rows, as the many-row kernel's (one per
// row) do; either way a warp's stores and the join's loads are contiguous.
template <int D, bool BY_FOURS>
__device__ __forceinline__ int64_t share_at(int64_t slot, int slot_rows, int row, int d) {
  return BY_FOURS ? ((slot * (D / 4) + d / 4) * slot_rows + row) * 4 : (slot * slot_rows + row) * D + d;
}

// Units [begin, end) of a split item: U per thread at a time, each by `lanes` lanes over the
// shares, whose loads are issued BATCH at a time.
template <int D, bool BY_FOURS, int U, int BATCH>
__device__ __forceinline__ void join_units(const TreeAttnArgs &a, const Share &s, int begin, int end, int lanes,
                                           int slot_rows, int tb) {
  const idx_tree_problem &p = a.p;
  const int G = p.Hq / p.cache.Hkv;
  const int sub = (threadIdx.x & 31) & (lanes - 1);
  const int step = 256 / lanes;
  for (int u0 = begin; u0 < end; u0 += U * step) {
    int row[U], d[U], prow[U];
    bool live[U];
    float m[U], l[U];
    float4 acc[U];
#pragma unroll
    for (int z = 0; z < U; ++z) {
      const int u = u0 + z * step + static_cast<int>(threadIdx.x) / lanes;
      live[z] = u < end;
      row[z] = d[z] = 0;
      if (live[z] && BY_FOURS) {
        d[z] = u / s.nrow;
        row[z] = u - d[z] * s.nrow;
        d[z] *= 4;
      } else if (live[z]) {
        row[z] = u / (D / 4);
        d[z] = (u - row[z] * (D / 4)) * 4;
      }
      prow[z] = a.pair && row[z] >= tb * G ? 128 + row[z] - tb * G : row[z];
      m[z] = -INFINITY;
      l[z] = 0.0f;
      acc[z] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int c0 = sub; c0 < s.count; c0 += BATCH * lanes) {
      float2 ml[U][BATCH];
      float4 o[U][BATCH];
#pragma unroll
      for (int z = 0; z < U; ++z)
#pragma unroll
        for (int y = 0; y < BATCH; ++y) {
          const int c = c0 + y * lanes;
          ml[z][y] = make_float2(-INFINITY, 0.0f);
          o[z][y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (!live[z] || c >= s.count) continue;
          const int64_t slot = c == 0 ? s.slot0 : 2 * (s.c0 + c);
          ml[z][y] = __ldcg(&a.part_ml[slot * slot_rows + prow[z]]);
          o[z][y] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + share_at<D, BY_FOURS>(slot, slot_rows, prow[z], d[z])));
        }
#pragma unroll
      for (int z = 0; z < U; ++z)
#pragma unroll
        for (int y = 0; y < BATCH; ++y) {
          const float nm = fmaxf(m[z], ml[z][y].x);
          const float f = ml[z][y].x == -INFINITY ? 0.0f : ex2(ml[z][y].x - nm), keep = m[z] == -INFINITY ? 0.0f : ex2(m[z] - nm);
          m[z] = nm;
          // a share that a row sees nothing of is 0; one whose weight vanishes is not left out: its
          // O may be NaN
          l[z] = l[z] * keep + f * ml[z][y].y;
          acc[z].x = acc[z].x * keep + f * o[z][y].x;
          acc[z].y = acc[z].y * keep + f * o[z][y].y;
          acc[z].z = acc[z].z * keep + f * o[z][y].z;
          acc[z].w = acc[z].w * keep + f * o[z][y].w;
        }
    }
#pragma unroll
    for (int z = 0; z < U; ++z) {
      float top = m[z];
      for (int o = lanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float f = m[z] == -INFINITY ? 0.0f : ex2(m[z] - top);
      float v[5] = {l[z], acc[z].x, acc[z].y, acc[z].z, acc[z].w};
#pragma unroll
      for (int y = 0; y < 5; ++y) v[y] *= f;
      for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int y = 0; y < 5; ++y) v[y] += __shfl_xor_sync(0xffffffffu, v[y], o);
      if (!live[z] || sub != 0) continue;
      const float inv = v[0] == 0.0f ? 0.0f : 1.0f / v[0];
      const int tok = row[z] / G;
      const int64_t at = static_cast<int64_t>(s.row0 + tok) * p.Hq + s.head * G + row[z] - tok * G;
      *reinterpret_cast<uint2 *>(a.out + at * D + d[z]) =
          make_uint2(pack_bf16(v[1] * inv, v[2] * inv), pack_bf16(v[3] * inv, v[4] * inv));
      if (d[z] == 0 && a.lse != nullptr) a.lse[at] = v[0] == 0.0f ? -INFINITY : (top + log2f(v[0])) * kLn2;
    }
  }
}

// Called by the 256 softmax threads of a CTA once its shares are written (thread 0's list).
template <int D, bool BY_FOURS>
__device__ __forceinline__ void join_items(const TreeAttnArgs &a, const Share *shares, const int *count, bool ok) {
  const idx_tree_problem &p = a.p;
  constexpr int kBatch = 8;   // shares whose loads are in flight together
  const int G = p.Hq / p.cache.Hkv;
  const int slot_rows = a.pair ? 256 : 128;
  const int tb = a.pair ? a.item_tokens / 2 : a.item_tokens;
  asm volatile("barrier.cta.sync 3, 256;" ::: "memory");
  const int n = *count;
  if (n == 0) return;
  if (threadIdx.x == 0) {
    __threadfence();
    for (int x = 0; x < n; ++x) atomicAdd(&a.joins[shares[x].c0].x, 1u);
    const uint64_t t0 = global_ns();
    for (int x = 0; x < n && ok; ++x) {
      volatile uint32_t *const in = &a.joins[shares[x].c0].x;
      while (*in < static_cast<uint32_t>(shares[x].count)) {
        if (global_ns() - t0 > a.wait_limit_ns) {
          flag_status(a.status, kStatusTimeout);
          break;
        }
      }
    }
    __threadfence();
  }
  asm volatile("barrier.cta.sync 3, 256;" ::: "memory");
  for (int x = 0; x < n; ++x) {
    const Share s = shares[x];
    const int k = static_cast<int>(blockIdx.x) - s.c0;
    const int units = s.nrow * (D / 4);       // of four values
    const int begin = static_cast<int>(static_cast<int64_t>(units) * k / s.count);
    const int end = static_cast<int>(static_cast<int64_t>(units) * (k + 1) / s.count);
    // lanes per unit, over the shares: as many as the units leave of the 256 threads
    int lanes = 1;
    while (lanes < 32 && 2 * lanes * (end - begin) <= 256) lanes *= 2;
    if (BY_FOURS && s.count <= kBatch / 2)   // few shares of many rows: two units at a time keep as many loads in flight
      join_units<D, BY_FOURS, 2, kBatch / 2>(a, s, begin, end, 1, slot_rows, tb);
    else
      join_units<D, BY_FOURS, 1, kBatch>(a, s, begin, end, lanes, slot_rows, tb);
  }
  // the last CTA out leaves the counters at zero for the next launch
  if (threadIdx.x == 0)
    for (int x = 0; x < n; ++x)
      if (atomicAdd(&a.joins[shares[x].c0].y, 1u) + 1u == static_cast<uint32_t>(shares[x].count)) {
        a.joins[shares[x].c0].x = 0u;
        a.joins[shares[x].c0].y = 0u;
      }
}

template <typename... Params, typename... Args>
cudaError_t launch_cooperative(void (*kernel)(Params...), int ctas, int threads, int smem, cudaStream_t stream,
                               Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace idx
