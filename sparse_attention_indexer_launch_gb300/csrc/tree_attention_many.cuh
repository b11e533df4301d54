// Attention of drafted tokens over a paged cache, whole or at selected positions, for more
// than 64 query vectors per key/value head and item.
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
// E4M3 keys feed the tensor core as they are: a row of Q, scaled by a power of two to
// at most 448, is split into two E4M3 terms whose sum it is (exactly, for elements down
// to 2^-9 of the row's largest; to 2^-17 of that below), and S is the sum of both
// terms' products.  P needs bf16's range (two E4M3 terms would drop what lies below
// 2^-18 of the largest, which adds up over a long cache), so V is converted to bf16 in
// shared memory, exactly.
//
// Work: an item is (request, key/value head, block of tokens) with its tiles in
// position order; the launch's tiles, in item order, are dealt out as one even,
// contiguous share per CTA (one CTA per SM).  A CTA that holds a whole item writes
// its output; shares of an item go to the state as (O, m, l), and the CTAs that hold them
// join them in a fixed order, so equal calls give equal bits.
//
// Two streams fill the tensor core: the even and odd tiles of one row block (up to 128
// rows, joined in TMEM at the end of the item) or two row blocks over the same tiles (more rows: each K and V
// tile is read from shared memory for 256 rows).  Each has O and two S buffers of 64
// columns in TMEM, so that the scores of a tile are computed while its four softmax
// warps, one thread per row, work on the tile before; P takes its S's place.
//
// What bounds it.  One row block: memory (8 requests' 16-node trees, 128 rows, over up to
// 256K bf16 keys 373 us, 6.2 TB/s).  Two: the softmax, at about 1,300 cycles for a tile of 64
// keys whose products take the tensor core as long, and the ends of items split over CTAs
// (4 requests' 64-node trees, 4,096 rows per request, 184.5 us, 1.0 PFLOP/s; 2 requests of
// 64 x 64 rows over 30,000 E4M3 keys of 2 heads 225 us).
#pragma once

#include "tree_attention_common.cuh"

namespace idx {
namespace {

constexpr int kTile = kPage;             // keys per tile
constexpr int kRows = 128;               // rows of a stream
constexpr uint32_t kColS = 0, kColO = 256;   // + 128 * stream (S: + 64 * buffer)

// ---------------------------------------------------------------------------- roles
// warps 0-3 and 4-7: softmax of streams 0 and 1; 8 and 11: loads of K and of V (by TMA,
// or gathering selected positions); 9 and 10: MMA issuers of streams 0 and 1; 12-19 with
// an E4M3 cache: the split of Q, and V to bf16, two teams of four on alternate loads; 13
// and 14 with two bf16 row blocks: issuers of the streams' scores.
constexpr int kKWarp = 8, kIssuerWarp = 9, kVWarp = 11, kConvertWarp = 12, kScoreWarp = 13;
constexpr int kMaxStages = 8;

// PAIR: two row blocks.
template <int D, bool F8, bool PAIR, bool SEL>
struct Cfg {
  static constexpr int kLoad = 128 / D;                  // pages per load of K or V
  static constexpr int kLoadBytes = kLoad * kTile * D * 2;   // as bf16
  static constexpr int kRawBytes = kLoad * kTile * D;        // as E4M3 bytes
  static constexpr int kKBytes = F8 ? kRawBytes : kLoadBytes;
  // Q of a row block: bf16, or the two E4M3 terms
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kQBufs = PAIR ? 1 : 2;
  static constexpr int kQTotal = kQBytes * (PAIR ? 2 : kQBufs);
  // The streams (and the converting teams) take alternate loads, so the counts are even: a
  // stage then always has the same waiter.  Were they odd, a waiter could come to a stage
  // again before the other's load in between, and the parity of the barrier would pass for
  // the one that it waits for.
  static constexpr int kKStages = F8 ? 6 : 4;
  static constexpr int kVStages = F8 ? 4 : D == 128 ? 4 : 6;      // as bf16
  static constexpr int kRawStages = F8 ? (D == 128 ? 4 : 6) : 0;  // V as E4M3
  static_assert(kKStages % 2 == 0 && kVStages % 2 == 0 && kRawStages % 2 == 0, "one waiter per stage");
  static constexpr int kScaleStages = F8 ? 8 : 0;
  static constexpr int kScaleFloats = 2 * kLoad * kTile;   // of a load: K's, then V's
  // Two row blocks keep an issuing thread busier than their softmax (a tcgen05.mma takes
  // it some 70 cycles): the scores' products then have threads of their own, in four more
  // warps (beside an E4M3 cache there are no registers for them).
  static constexpr bool kSplitIssue = PAIR && !F8;
  static constexpr int kThreads = 32 * (F8 ? kConvertWarp + 8 : kSplitIssue ? kConvertWarp + 4 : kConvertWarp);
  // Registers per thread after the roles part, where a softmax thread holds up to 64
  // scores.  The shares add up to no more than the launch's threads x registers.
  static constexpr bool kShareRegs = kThreads > 384;
  static constexpr int kRegsLaunch = F8 ? 96 : 128, kRegsSoftmax = F8 ? 144 : 176, kRegsOther = F8 ? 64 : 80;
  static_assert(!kShareRegs || 256 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * kRegsLaunch, "register shares");
  static constexpr int kDynamic = 1024 + kQTotal + kKStages * kKBytes + kVStages * kLoadBytes + kRawStages * kRawBytes +
                                  kScaleStages * kScaleFloats * 4;
};

template <bool PAIR>
struct Barriers {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t raw_full[kMaxStages], raw_empty[kMaxStages];
  uint64_t sc_full[kMaxStages], sc_empty[kMaxStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2];   // [stream][buffer]
  uint64_t o_free[2], drain[2], drain_s[2], scrubbed[2];
  // [stream][segment parity]: a stream without tiles in a segment may be one segment ahead
  uint64_t stats[2][2];
  uint32_t tmem_base;
  int abort;
  int32_t two_terms[2][2];         // P of [stream][buffer] has a low term
  Start found;                     // the share's first request
  Share shares[2];                 // of split items
  int nshare;                      // how many there are
  uint32_t page_ok[64], vpage_ok[64];   // dense: the page of tile k % 64 of the CTA was loaded (K, V)
  uint32_t keys_ok[64][2];         // selected: bit per key of tile k % 64
  int32_t nonfinite[32];           // segment number + 1 whose drafted tokens' V held NaN or infinity
  float row_m[PAIR ? 1 : 2][2][PAIR ? 1 : kRows], row_l[PAIR ? 1 : 2][2][PAIR ? 1 : kRows];   // [segment parity][stream][row]
  // E4M3: 1 / the row's power of two, [segment % 4][row block][row].  Q of a segment is split
  // at most three segments before the softmax has begun with it: S of the second next one
  // takes the place of P of this one.
  float q_scale[4][PAIR ? 2 : 1][kRows];
  int warp_sums[20];
};

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
  tc_fence_after();   // the product's O, before it is read
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

// One row's keys of a tile: S (64 columns at ts) to P in the same columns, the row's maximum
// m and sum l, and O (D columns at to) when the maximum moves.  special: only the keys of ok
// (a bit per key) are visible.  sk: the tile's K scales; sv: its V scales.
//
// P is rounded to bf16 for the product with V.  That leaves an error nearly as large as the
// output's own rounding (relative to the output 0.9e-3 over 128 keys to 1.5e-3 over 65,536,
// beside 1.7e-3), for half the products that two terms would take.  The few visible keys of a
// special tile average out less (up to 2^-8 of one value): there P is kept in two bf16 terms,
// high in columns 0-31 and low in 32-63, and the product runs over both.
template <int D, bool F8, typename F>
__device__ __forceinline__ bool softmax_tile(uint32_t ts, uint32_t to, const float *sk, const float *sv, float c, bool special,
                                             uint64_t ok, bool has_o, float &m, float &l, F settled) {
  constexpr int kW = 32;        // columns per register group
  uint32_t x[2][kW];
#pragma unroll
  for (int w = 0; w < 2; ++w) tmem_ld32(ts + 32 * w, x[w]);
  const float4 *const ks = reinterpret_cast<const float4 *>(sk);
  const float2 *const vs = reinterpret_cast<const float2 *>(sv);
  tmem_wait_ld();
#pragma unroll
  for (int w = 0; w < 2; ++w) reg_fence32(x[w]);
  if (F8) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
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
    if (c == 0.0f) {   // scores of 0 (or NaN): multiplied here, so that what is masked below stays -infinity
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int y = 0; y < kW; ++y) x[w][y] = __float_as_uint(__uint_as_float(x[w][y]) * c);
      c = 1.0f;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int y = 0; y < kW; ++y)
        x[w][y] = (static_cast<uint32_t>(ok >> (32 * w)) >> y) & 1u ? x[w][y] : 0xFF800000u;   // -infinity
  }
  float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int y = 0; y < kW; y += 8)
#pragma unroll
      for (int z = 0; z < 4; ++z)
        t4[z] = max3(t4[z], __uint_as_float(x[w][y + 2 * z]), __uint_as_float(x[w][y + 2 * z + 1]));
  const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c;   // in units of log2
  if (!raise_maximum<D>(to, top, has_o, m, l, settled)) return false;
  const float base = m == -INFINITY ? 0.0f : m;
  const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
  float2 l2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int w = 0; w < 2; ++w) {
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
    tmem_st16(ts + 16 * w, hi);
    if (special) {
      uint32_t lo[kW / 2];
#pragma unroll
      for (int y = 0; y < kW / 2; ++y) {
        // an infinity (a scale's) has no low term
        const float r0 = __uint_as_float(x[w][2 * y]) - __uint_as_float(hi[y] << 16);
        const float r1 = __uint_as_float(x[w][2 * y + 1]) - __uint_as_float(hi[y] & 0xFFFF0000u);
        lo[y] = pack_bf16(r0 == r0 ? r0 : 0.0f, r1 == r1 ? r1 : 0.0f);
      }
      tmem_st16(ts + 32 + 16 * w, lo);
    }
  }
  l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
  tmem_wait_st();
  return true;
}

// ---------------------------------------------------------------------------- kernel
template <int D, bool F8, bool PAIR, bool SEL>
__global__ void __launch_bounds__(Cfg<D, F8, PAIR, SEL>::kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const TreeAttnArgs a) {
  using C = Cfg<D, F8, PAIR, SEL>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Barriers<PAIR> bars;
  uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  uint8_t *const sq = smem;
  uint8_t *const sk = sq + C::kQTotal;
  uint8_t *const sv = sk + C::kKStages * C::kKBytes;
  uint8_t *const sraw = sv + C::kVStages * C::kLoadBytes;
  float *const ssc = reinterpret_cast<float *>(sraw + C::kRawStages * C::kRawBytes);   // [stage][K, V]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const idx_tree_problem &p = a.p;
  const int Hkv = p.cache.Hkv;
  const int G = p.Hq / Hkv;
  const int tb = PAIR ? a.item_tokens / 2 : a.item_tokens;   // tokens of a row block
  constexpr int kBlocks = D / 64;            // 64-dimension blocks of a bf16 operand
  constexpr int kLoad = C::kLoad;            // tiles per load
  constexpr int kBlockBytes = kLoad * kTile * 128, kQBlockBytes = kRows * 128;

  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.k_empty[s], PAIR ? 2 : 1);
      mbar_init(&bars.v_full[s], F8 ? 4 : 1);    // by a team's four warps, or the loading one
      mbar_init(&bars.v_empty[s], PAIR ? 2 : 1);
      mbar_init(&bars.raw_full[s], 1);
      mbar_init(&bars.raw_empty[s], 4);
      mbar_init(&bars.sc_full[s], 2);            // K's and V's scales
      mbar_init(&bars.sc_empty[s], PAIR ? 8 : 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.q_full[s], F8 ? 8 : 1);
      mbar_init(&bars.q_empty[s], 2);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars.s_full[s][b], 1);
        mbar_init(&bars.p_ready[s][b], 4);
        mbar_init(&bars.pv_done[s][b], 1);
      }
      mbar_init(&bars.o_free[s], PAIR ? 4 : 8);
      mbar_init(&bars.drain[s], 1);
      mbar_init(&bars.drain_s[s], 1);
      for (int b = 0; b < 2; ++b) mbar_init(&bars.stats[s][b], 4);
      mbar_init(&bars.scrubbed[s], 4);
    }
    bars.abort = 0;
    bars.nshare = 0;
    for (int s = 0; s < 32; ++s) bars.nonfinite[s] = 0;
    fence_barrier_init();
  }
  if (warp == kIssuerWarp) {
    tmem_alloc(&bars.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (tid == kKWarp * 32) {
    if (!F8) prefetch_tensormap(&qmap);
    if (!SEL) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
  }

  const Start start = find_share<C::kThreads>(a, &bars.found, bars.warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const Shares share(start.W, a.tile, gridDim.x);
  const bool idle = static_cast<int>(blockIdx.x) >= share.n || start.W == 0;
  const int t0 = idle ? 0 : share.begin(blockIdx.x), t1 = idle ? 0 : share.begin(blockIdx.x + 1);
  const Start &first = p.Q > 32 && !idle ? bars.found : start;
  Walk walk(a, t0, t1, first.req, first.base, first.q);

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
    const int s = warp >> 2;               // stream
    const int row = tid & 127;             // row of the stream's tile, and its TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // first TMEM lane of the warp << 16
    const uint32_t to = tmem + kColO + 128 * s + lanes;
    const float c = p.scale * kLog2e;
    const int step = PAIR ? 1 : 2;
    int tiles = 0;      // tiles of earlier segments
    int loads = 0;      // loads of earlier segments
    uint32_t n = 0;     // this stream's tiles so far
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
      const int j0 = PAIR ? 0 : (s ^ loads) & 1;   // the stream's first load: the CTA's even or odd ones
      float cs = c;      // of the row's scores
      for (int jj = j0; ok && live && jj * kLoad < walk.count; jj += step)
      for (int j = jj * kLoad; j < min(walk.count, (jj + 1) * kLoad); ++j, ++n, ++mine) {
        const int k = tiles + j, ld = loads + jj, sub = j - jj * kLoad;
        const int key0 = (walk.tile0 + j) * kTile;
        const int buf = n & 1;
        if ((F8 && sub == 0 && !warp_wait_all(&bars.sc_full[ld % 8], (ld / 8) & 1)) ||
            !warp_wait_all(&bars.s_full[s][buf], (n >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (F8 && mine == 0) cs = c * bars.q_scale[walk.seg & 3][PAIR ? s : 0][row];
        uint64_t okbits = ~0ull;   // keys of the tile that the row sees
        bool special;
        if (SEL) {
          const uint32_t k0 = bars.keys_ok[k & 63][0], k1 = bars.keys_ok[k & 63][1];
          special = (k0 & k1) != ~0u;
          if (special) okbits = static_cast<uint64_t>(k1) << 32 | k0;
        } else {
          const uint32_t page = bars.page_ok[k & 63];
          special = key0 + kTile > ctx || page == 0u;
          if (special) {
            const int lim = walk.q.keys - ctx;      // drafted tokens within the page table
            const uint64_t vm = lim >= 64 ? mask : mask & ((1ull << lim) - 1ull);
            const int before = ctx - key0;          // cached keys from the tile's first on
            if (before < 64) {
              if (before > 0) okbits = ((1ull << before) - 1ull) | (vm << before);
              else okbits = before > -64 ? vm >> -before : 0ull;
            }
            if (page == 0u) okbits = 0ull;
          }
        }
        if (!SEL && !F8 && special) {
          // V of tokens that some rows do not see has to be finite (0 x NaN is NaN): zero
          // what no row sees, and what is not finite among the drafted tokens (rows that
          // see it get it back at the end).  Two threads share a key.
          const int sl = ld % C::kVStages;
          if (!warp_wait_all(&bars.v_full[sl], (ld / C::kVStages) & 1)) {
            ok = false;
            break;
          }
          const int key = row & 63, pos = key0 + key;
          const bool dead = pos >= walk.q.keys || bars.page_ok[k & 63] == 0u;
          if (dead || pos >= ctx) {
#pragma unroll 4
            for (int x = (row >> 6) * kBlocks * 4; x < (row >> 6) * kBlocks * 4 + kBlocks * 4; ++x) {
              uint4 *const at = reinterpret_cast<uint4 *>(sv + sl * C::kLoadBytes + (x >> 3) * kBlockBytes +
                                                          (sub * kTile + key) * 128 + ((x + key) & 7) * 16);
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
          const float *const ks = ssc + (ld % 8) * C::kScaleFloats + sub * kTile;
          if (!softmax_tile<D, F8>(tmem + kColS + 128 * s + 64 * buf + lanes, to, ks, ks + kLoad * kTile, cs,
                                   special, okbits, mine > 0, m, l, settled)) {
            ok = false;
            break;
          }
        }
        if (row == 0) bars.two_terms[s][buf] = special;
        tc_fence_before();
        warp_arrive(&bars.p_ready[s][buf]);
        if (F8 && lane == 0 && (sub == kLoad - 1 || j + 1 == walk.count)) mbar_arrive(&bars.sc_empty[ld % 8]);
      }
      if (!ok) break;
      if (F8 && PAIR && !live)   // hand the scales of the tiles on
        for (int jj = 0; jj * kLoad < walk.count; ++jj) {
          const int ld = loads + jj;
          if (!warp_wait_all(&bars.sc_full[ld % 8], (ld / 8) & 1)) {
            ok = false;
            break;
          }
          warp_arrive(&bars.sc_empty[ld % 8]);
        }
      if (!ok) break;
      const int odd = loads & 1, nloads = (walk.count + kLoad - 1) / kLoad;
      const bool has0 = PAIR || odd < nloads, has1 = !PAIR && (odd ^ 1) < nloads;   // the streams that had tiles
      tiles += walk.count;
      loads += nloads;

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
      if constexpr (!PAIR) {
        // the row's maximum and sum over both streams, whose O scale by f0 and f1
        const int sp = walk.seg & 1;
        bars.row_m[sp][s][row] = m;
        bars.row_l[sp][s][row] = l;
        tc_fence_before();
        warp_arrive(&bars.stats[s][sp]);
        if (!warp_wait_all(&bars.stats[s][sp], (walk.seg >> 1) & 1) ||
            !warp_wait_all(&bars.stats[s ^ 1][sp], (walk.seg >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float m0 = bars.row_m[sp][0][row], m1 = bars.row_m[sp][1][row], mm = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.0f : ex2(m0 - mm);
        f1 = m1 == -INFINITY ? 0.0f : ex2(m1 - mm);
        l = bars.row_l[sp][0][row] * f0 + bars.row_l[sp][1][row] * f1;
        m = mm;
      }
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
          *reinterpret_cast<float4 *>(a.part_o + share_at<D, true>(slot, kSlotRows, prow, d)) = o;
        }
      };
      if (row < nrow && (PAIR || s == 0)) {
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
          if (has0) tmem_ld16(o0 + d, x);
          if (has1) tmem_ld16(o0 + 128 + d, x1);
          tmem_wait_ld();
          reg_fence16(x);
          reg_fence16(x1);
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            o[y] = PAIR ? __uint_as_float(x[y]) : has0 ? __uint_as_float(x[y]) * f0 : 0.0f;
            if (has1) o[y] += __uint_as_float(x1[y]) * f1;
          }
        }
        if (row < nrow)
#pragma unroll
          for (int y = 0; y < 16; y += 4) put(d + y, make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.o_free[PAIR ? s : 0]);
        if (!PAIR) mbar_arrive(&bars.o_free[1]);
      }
      if (!walk.whole && tid == 0) bars.shares[bars.nshare++] = share_of(walk, share, G);
    }
    if (!ok) give_up();
    join_items<D, true>(a, bars.shares, &bars.nshare, ok);
  } else if (warp < kConvertWarp || C::kSplitIssue) {
    if constexpr (C::kShareRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kKWarp || warp == kVWarp) {
      // -------------------------------------------------------------- loads
      // K's warp also brings a bf16 Q; each brings its own scales.
      const bool is_v = warp == kVWarp;
      const int stages = is_v ? (F8 ? C::kRawStages : C::kVStages) : C::kKStages;
      const int bytes = is_v ? (F8 ? C::kRawBytes : C::kLoadBytes) : C::kKBytes;
      uint64_t *const full = is_v ? (F8 ? bars.raw_full : bars.v_full) : bars.k_full;
      uint64_t *const empty = is_v ? (F8 ? bars.raw_empty : bars.v_empty) : bars.k_empty;
      uint8_t *const ring = is_v ? (F8 ? sraw : sv) : sk;
      const float *const scales = is_v ? p.cache.v_scale : p.cache.k_scale;
      float *const sscale = ssc + (is_v ? kLoad * kTile : 0);
      int stage = 0;          // of the next load
      uint32_t phase = 1;     // its empty barrier's
      int nload = 0;          // loads so far
      int tiles = 0;          // tiles of earlier segments
      int nq = 0;             // Q loads so far
      bool ok = true;
      auto warp_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        int r = 1;
        if (lane == 0) r = mbar_wait(bar, parity, limit, abort);
        return __shfl_sync(0xffffffffu, r, 0) != 0;
      };
      // Gathering: copies of up to kPend loads stay in flight while the next is issued;
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
        const int nloads = (walk.count + kLoad - 1) / kLoad;
        if (!F8 && !is_v) {
          const int qb = walk.seg % C::kQBufs;
          if (!wait_flushed(&bars.q_empty[qb], ((walk.seg / C::kQBufs) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const int nhalf = PAIR && walk.tokens > tb ? 2 : 1;
            mbar_arrive_expect_tx(&bars.q_full[qb], static_cast<uint32_t>(nhalf * kBlocks * G * tb * 128));
            for (int s = 0; s < nhalf; ++s)
              for (int b = 0; b < kBlocks; ++b)
                tma_load_3d(sq + (PAIR ? s : qb) * C::kQBytes + b * kQBlockBytes, &qmap, b * 64, walk.head * G,
                            walk.q.row0 + walk.tok0 + s * tb, &bars.q_full[qb]);
          }
          ++nq;
        }
        const int32_t *const table = p.page_table + static_cast<int64_t>(walk.i) * p.pt_stride;
        if constexpr (SEL) {
          // ---------------------------------------------------------- gathering
          const int r = walk.q.row0 + walk.tok0;
          const uint64_t mask = p.mask != nullptr ? p.mask[r] : (2ull << walk.tok0) - 1ull;
          const int32_t *const sel = a.sel + static_cast<int64_t>(r) * a.sel_k;
          const int n0 = walk.tile0 * kTile + lane, nend = n0 - lane + walk.count * kTile;
          constexpr int kPer = 2 * kLoad;      // keys of a load per lane: lane, lane + 32 ..
          // A key's way: its entry of the selection, its page, its slot; each step's load is
          // issued a load or more ahead of the next step, so that none is waited for.
          auto entry = [&](int jj, int x) -> int32_t {
            const int n = n0 + (jj * kPer + x) * 32;
            return n < nend && n < a.sel_k ? sel[n] : -1;
          };
          auto position = [&](int jj, int x, int32_t e) -> int32_t {   // logical position, -1 for none
            const int n = n0 + (jj * kPer + x) * 32;
            if (n >= nend) return -1;
            if (n < a.sel_k) return e >= 0 && e < walk.q.ctx ? e : -1;
            const int u = n - a.sel_k;
            return u < walk.q.tokens && ((mask >> u) & 1ull) && walk.q.ctx + u < walk.q.keys ? walk.q.ctx + u : -1;
          };
          auto page_of = [&](int32_t pos) -> int32_t { return pos >= 0 ? table[pos / kPage] : -1; };
          int32_t pos[2][kPer], pg[2][kPer], e[3][kPer];   // loads jj, jj + 1; jj + 2 .. jj + 4
#pragma unroll
          for (int x = 0; x < kPer; ++x) {
            pos[0][x] = entry(0, x);
            pos[1][x] = entry(1, x);
#pragma unroll
            for (int y = 0; y < 3; ++y) e[y][x] = entry(2 + y, x);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
              pos[y][x] = position(y, x, pos[y][x]);
              pg[y][x] = page_of(pos[y][x]);
            }
          for (int jj = 0; jj < nloads; ++jj) {
            if (!wait_flushed(&empty[stage], phase)) {
              ok = false;
              break;
            }
            if (F8 && !wait_flushed(&bars.sc_empty[nload % 8], ((nload / 8) & 1) ^ 1)) {
              ok = false;
              break;
            }
            uint8_t *const dst = ring + stage * bytes;
            float *const dsc = sscale + (nload % 8) * C::kScaleFloats;
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
              int32_t slot = -1;           // page * 64 + token
              if (pos[0][x] >= 0) {
                if (pg[0][x] >= 0 && pg[0][x] < p.cache.P) slot = pg[0][x] * kPage + pos[0][x] % kPage;
                else flag_status(a.status, kStatusBadPage);
              }
              const uint32_t bits = __ballot_sync(0xffffffffu, slot >= 0);
              if (!is_v && lane == 0) bars.keys_ok[(tiles + jj * kLoad + x / 2) & 63][x & 1] = bits;
              const int64_t off = slot < 0 ? -1
                                           : (static_cast<int64_t>(slot / kPage) * p.cache.page_stride +
                                              (slot % kPage) * p.cache.token_stride + walk.head * p.cache.head_stride) *
                                                 (F8 ? 1 : 2);
              if constexpr (F8) {
                const int64_t at = slot < 0 ? 0
                                            : (static_cast<int64_t>(slot / kPage) * Hkv + walk.head) * kPage + slot % kPage;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dsc + x * 32 + lane)),
                             "l"(scales + at), "r"(slot < 0 ? 0 : 4)
                             : "memory");
              }
              // 16 bytes per lane: D / 16 or D / 8 lanes bring one key
              constexpr int kLanes = F8 ? D / 16 : D / 8;
              constexpr int kKeysAtOnce = 32 / kLanes;
              const uint8_t *const cache = static_cast<const uint8_t *>(is_v ? p.cache.v : p.cache.k);
              const int ch = lane % kLanes;
#pragma unroll
              for (int y = 0; y < kLanes; ++y) {
                const int from = y * kKeysAtOnce + lane / kLanes;
                const int64_t o = __shfl_sync(0xffffffffu, off, from);
                const int key = x * 32 + from;
                uint32_t at;   // bf16: blocks of 128-byte rows, swizzled; E4M3 K: rows of D, swizzled; V: rows of D
                if (!F8) at = (ch >> 3) * kBlockBytes + key * 128 + (((ch & 7) ^ (key & 7)) << 4);
                else if (is_v) at = key * D + ch * 16;
                else at = key * D + ((D == 128 ? ch ^ (key & 7) : ch ^ ((key >> 1) & 3)) << 4);
                const uint8_t *const src = cache + (o < 0 ? 0 : o) + ch * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst) + at), "l"(src),
                             "r"(o < 0 ? 0 : 16)
                             : "memory");
              }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group %0;" ::"n"(kPend) : "memory");
            landed(0);
#pragma unroll
            for (int x = 0; x + 1 < kPend; ++x) {
              pend[x] = pend[x + 1];
              pend_sc[x] = pend_sc[x + 1];
            }
            pend[kPend - 1] = &full[stage];
            pend_sc[kPend - 1] = F8 ? &bars.sc_full[nload % 8] : nullptr;
            ++nload;
            if (++stage == stages) {
              stage = 0;
              phase ^= 1u;
            }
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
              pos[0][x] = pos[1][x];
              pg[0][x] = pg[1][x];
              pos[1][x] = position(jj + 2, x, e[0][x]);
              pg[1][x] = page_of(pos[1][x]);
              e[0][x] = e[1][x];
              e[1][x] = e[2][x];
              e[2][x] = entry(jj + 5, x);
            }
          }
        } else {
          // ---------------------------------------------------------- pages by TMA
          const void *const map = is_v ? &vmap : &kmap;
          uint32_t *const oks = is_v ? bars.vpage_ok : bars.page_ok;
          // page ids of 32 tiles of the segment at a time (tiles are pages)
          auto fetch = [&](int j) -> int32_t { return j + lane < walk.count ? table[walk.tile0 + j + lane] : -2; };
          int32_t ids = fetch(0), ids_next = fetch(32);
          for (int jj = 0; jj < nloads; ++jj) {
            const int j = jj * kLoad;
            if (j > 0 && (j & 31) == 0) {
              ids = ids_next;
              ids_next = fetch(j + 32);
            }
            int32_t pg[kLoad];
            uint32_t good = 0;
#pragma unroll
            for (int x = 0; x < kLoad; ++x) {
              pg[x] = __shfl_sync(0xffffffffu, ids, (j + x) & 31);
              good += pg[x] >= 0 && pg[x] < p.cache.P;
            }
            if (!warp_wait(&empty[stage], phase) ||
                (F8 && !warp_wait(&bars.sc_empty[nload % 8], ((nload / 8) & 1) ^ 1))) {
              ok = false;
              break;
            }
            if (lane == 0) {
              uint8_t *const dst = ring + stage * bytes;
              if (good == kLoad) {
                mbar_arrive_expect_tx(&full[stage], bytes);
              } else {
                mbar_arrive_expect_tx(&full[stage], good * static_cast<uint32_t>(bytes / kLoad));
              }
              if (F8) mbar_arrive_expect_tx(&bars.sc_full[nload % 8], good * 256u);
#pragma unroll
              for (int x = 0; x < kLoad; ++x) {
                const bool there = pg[x] >= 0 && pg[x] < p.cache.P;
                oks[(tiles + j + x) & 63] = there;
                if (!there) {
                  if (pg[x] != -2) flag_status(a.status, kStatusBadPage);
                  continue;
                }
                if constexpr (F8) {
                  tma_load_4d(dst + x * (kTile * D), map, 0, 0, walk.head, pg[x], &full[stage]);
                  bulk_load(sscale + (nload % 8) * C::kScaleFloats + x * kTile,
                            scales + (static_cast<int64_t>(pg[x]) * Hkv + walk.head) * kPage, 256u,
                            &bars.sc_full[nload % 8]);
                } else {
#pragma unroll
                  for (int b = 0; b < kBlocks; ++b)
                    tma_load_4d(dst + b * kBlockBytes + x * (kTile * 128), map, b * 64, 0, walk.head, pg[x], &full[stage]);
                }
              }
            }
            ++nload;
            if (++stage == stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        tiles += walk.count;
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
        land(bars.q_full, C::kQBufs, nq);
        if (!SEL) {
          land(full, stages, nload);
          if (F8) land(bars.sc_full, 8, nload);
        }
      }
    } else if (warp == kIssuerWarp || warp == kIssuerWarp + 1 || warp == kScoreWarp || warp == kScoreWarp + 1) {
      // -------------------------------------------------------------- MMA issuers
      // Per stream: S of two tiles; then, tile by tile, O += P V once its P is ready, and S
      // of the second next tile once that has completed, since it takes P's columns.  One
      // thread does both, or one each (the kScoreWarps S).
      if (lane == 0) {
        const int s = (warp - kIssuerWarp) & 1;
        static_assert((kScoreWarp - kIssuerWarp) % 2 == 0);
        const bool do_s = !C::kSplitIssue || warp >= kScoreWarp, do_pv = !C::kSplitIssue || warp < kScoreWarp;
        const uint32_t ts = tmem + kColS + 128 * s, to = tmem + kColO + 128 * s;
        const uint32_t idesc_s = umma_idesc(F8 ? 0u : 1u, kTile), idesc_o = umma_idesc(1u, D) | kIdescBMn;
        int kstage = 0, vstage = 0;          // of the next load of K and of V
        uint32_t kphase = 0, vphase = 0;
        uint32_t ns = 0;    // this stream's S so far
        uint32_t n = 0;     // this stream's products with V so far
        bool ok = true, any = false;
        auto skip = [&](int &stage, uint32_t &phase, int stages, int by) {
          stage += by;
          while (stage >= stages) {
            stage -= stages;
            phase ^= 1u;
          }
        };
        const int step = PAIR ? 1 : 2;
        int loads = 0;      // of earlier segments
        while (ok && walk.next()) {
          const int qb = walk.seg % C::kQBufs;
          const int nloads = (walk.count + kLoad - 1) / kLoad;
          const bool live = !PAIR || s == 0 || walk.tokens > tb;   // this stream has rows
          if (do_s && !mbar_wait(&bars.q_full[qb], (walk.seg / C::kQBufs) & 1, limit, abort)) {
            ok = false;
            break;
          }
          const int j0 = PAIR ? 0 : (s ^ loads) & 1;   // the stream's first load
          loads += nloads;
          if (do_s && j0 >= nloads) mbar_arrive(&bars.q_empty[qb]);
          // the stream's first load, and what lies before the next segment's
          skip(kstage, kphase, C::kKStages, j0);
          skip(vstage, vphase, C::kVStages, j0);
          if (!live) {   // no rows: only pass the loads on
            for (int jj = 0; ok && jj < nloads; ++jj) {
              ok = (!do_s || mbar_wait(&bars.k_full[kstage], kphase, limit, abort)) &&
                   (!do_pv || mbar_wait(&bars.v_full[vstage], vphase, limit, abort));
              if (!ok) break;
              if (do_s) mbar_arrive(&bars.k_empty[kstage]);
              if (do_pv) mbar_arrive(&bars.v_empty[vstage]);
              skip(kstage, kphase, C::kKStages, 1);
              skip(vstage, vphase, C::kVStages, 1);
            }
            if (ok && do_s) mbar_arrive(&bars.q_empty[qb]);
            continue;
          }
          const uint32_t qaddr = smem_u32(sq + (PAIR ? s : qb) * C::kQBytes);
          int jk = j0, subk = 0;               // the next S
          auto scores = [&]() -> bool {
            if (subk == 0 && !mbar_wait(&bars.k_full[kstage], kphase, limit, abort)) return false;
            tc_fence_after();
            const uint32_t d = ts + 64 * (ns & 1);
            const uint32_t kaddr = smem_u32(sk + kstage * C::kKBytes);
            if constexpr (F8) {
              // both terms of Q over the same keys: D = 128: 128-byte rows, the terms 16 KB
              // apart; D = 64: the terms side by side in 128-byte rows, keys in 64-byte rows
              const uint64_t qdesc = umma_desc_sw128(qaddr);
              const uint64_t kdesc = D == 128 ? umma_desc_sw128(kaddr) : umma_desc_sw64(kaddr + subk * kTile * 64);
#pragma unroll
              for (int kk = 0; kk < 2 * D / 32; ++kk) {
                const int term = kk / (D / 32), x = kk % (D / 32);
                umma_f8(d, qdesc + ((term * (D == 128 ? kQBlockBytes : 64) + x * 32) >> 4), kdesc + ((x * 32) >> 4),
                        idesc_s, kk > 0);
              }
            } else {
              const uint64_t qdesc = umma_desc_sw128(qaddr), kdesc = umma_desc_sw128(kaddr + subk * kTile * 128);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_f16(d, qdesc + (((kk >> 2) * kQBlockBytes + (kk & 3) * 32) >> 4),
                         kdesc + (((kk >> 2) * kBlockBytes + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
            }
            umma_commit(&bars.s_full[s][ns & 1]);
            any = true;
            ++ns;
            if (++subk == kLoad || jk * kLoad + subk == walk.count) {   // the load's last tile
              umma_commit(&bars.k_empty[kstage]);
              subk = 0;
              jk += step;
              skip(kstage, kphase, C::kKStages, jk < nloads ? step : 0);
              if (jk >= nloads) umma_commit(&bars.q_empty[qb]);
            }
            return true;
          };
          if (!do_pv) {
            // the product of the tile before the last has to have left the buffer
            while (ok && jk < nloads)
              ok = (ns < 2 || mbar_wait(&bars.pv_done[s][ns & 1], ((ns - 2) >> 1) & 1, limit, abort)) && scores();
            skip(kstage, kphase, C::kKStages, 1);   // to the next segment's first load
            continue;
          }
          if (do_s && jk < nloads) ok = scores();
          if (do_s && ok && jk < nloads) ok = scores();
          for (int jj = j0; ok && jj < nloads; jj += step) {
            const int end = min(walk.count, (jj + 1) * kLoad);
            for (int j = jj * kLoad; j < end; ++j, ++n) {
              const int buf = n & 1, sub = j - jj * kLoad;
              if (!mbar_wait(&bars.p_ready[s][buf], (n >> 1) & 1, limit, abort) ||
                  (j == j0 * kLoad && !mbar_wait(&bars.o_free[s], (walk.seg & 1) ^ 1, limit, abort)) ||
                  (sub == 0 && !mbar_wait(&bars.v_full[vstage], vphase, limit, abort))) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t vdesc = umma_desc_mn(smem_u32(sv + vstage * C::kLoadBytes + sub * kTile * 128), kBlockBytes);
              const uint32_t ta = ts + 64 * buf;
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                umma_f16_ta(to, ta + kk * 8, vdesc + ((kk * 2048) >> 4), idesc_o, j > j0 * kLoad || kk > 0);
              if (*reinterpret_cast<volatile int32_t *>(&bars.two_terms[s][buf])) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                  umma_f16_ta(to, ta + 32 + kk * 8, vdesc + ((kk * 2048) >> 4), idesc_o, 1u);
              }
              umma_commit(&bars.pv_done[s][buf]);
              any = true;
              if (j + 1 == end) {
                umma_commit(&bars.v_empty[vstage]);
                skip(vstage, vphase, C::kVStages, jj + step < nloads ? step : 0);
              }
              if (do_s) ok = mbar_wait(&bars.pv_done[s][buf], (n >> 1) & 1, limit, abort) && (jk >= nloads || scores());
              if (!ok) break;
            }
          }
          // to the next segment's first load
          const int left = j0 < nloads ? (nloads - j0 - 1) % step + 1 : 0;
          skip(kstage, kphase, C::kKStages, left);
          skip(vstage, vphase, C::kVStages, left);
        }
        if (!ok) {
          give_up();
          if (any) {   // MMAs in flight read shared memory and TMEM: wait for them
            uint64_t *const drain = do_pv ? &bars.drain[s] : &bars.drain_s[s];
            umma_commit(drain);
            if (!mbar_wait(drain, 0, limit, &never)) flag_status(a.status, kStatusTimeout);
          }
        }
      }
    }
  } else {
    if constexpr (F8) {
      // -------------------------------------------------------------- E4M3: Q split, V to bf16
      if constexpr (C::kShareRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
      const int team = (warp - kConvertWarp) >> 2, t = (tid - kConvertWarp * 32) & 127;
      Walk qwalk(a, t0, t1, first.req, first.base, first.q);     // the segment whose Q is next
      // Q of qwalk's segment: two threads per row (of every row block), each with half of
      // its dimensions.  Both terms go to shared memory, rows without a token as
      // zeros.
      auto split_q = [&]() -> bool {
        const int qb = qwalk.seg % C::kQBufs;
        if (!warp_wait_all(&bars.q_empty[qb], ((qwalk.seg / C::kQBufs) & 1) ^ 1)) return false;
        const int id = tid - kConvertWarp * 32, row = id >> 1, half = id & 1;
#pragma unroll 1
        for (int blk = 0; blk < (PAIR && qwalk.tokens > tb ? 2 : 1); ++blk) {
          const int nrow = min(tb, qwalk.tokens - blk * tb) * G;
          uint4 v[D / 16];
          const uint16_t *const src = static_cast<const uint16_t *>(p.q) +
                                      static_cast<int64_t>(qwalk.q.row0 + qwalk.tok0 + blk * tb + row / G) * p.q_row_stride +
                                      static_cast<int64_t>(qwalk.head * G + row % G) * D + half * (D / 2);
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            v[x] = row < nrow ? __ldg(reinterpret_cast<const uint4 *>(src) + x) : make_uint4(0, 0, 0, 0);
          // the row's largest exponent (of the finite elements: NaN and infinity stay what they are)
          uint32_t top = 0;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t lo = w[y] & 0x7FFFu, hi = (w[y] >> 16) & 0x7FFFu;
              if (lo < 0x7F80u) top = max(top, lo);
              if (hi < 0x7F80u) top = max(top, hi);
            }
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          // 2^e takes it to (224, 448]; rows below 2^-112 stop at 2^120
          const int e = min(((top & 0x7Fu) <= 0x60u ? 8 : 7) - (static_cast<int>(top >> 7) - 127), 120);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          if (half == 0)
            bars.q_scale[qwalk.seg & 3][PAIR ? blk : 0][row] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          uint8_t *const dst = sq + (PAIR ? blk : qb) * C::kQBytes;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {       // 16 elements: 16 bytes of each term
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t a0 = y < 2 ? (y == 0 ? v[2 * x].x : v[2 * x].z) : (y == 2 ? v[2 * x + 1].x : v[2 * x + 1].z);
              const uint32_t a1 = y < 2 ? (y == 0 ? v[2 * x].y : v[2 * x].w) : (y == 2 ? v[2 * x + 1].y : v[2 * x + 1].w);
              const float f0 = __uint_as_float(a0 << 16) * up, f1 = __uint_as_float(a0 & 0xFFFF0000u) * up;
              const float f2 = __uint_as_float(a1 << 16) * up, f3 = __uint_as_float(a1 & 0xFFFF0000u) * up;
              const uint32_t h0 = e4m3x2(f0, f1), h1 = e4m3x2(f2, f3);
              const float2 g0 = e4m3x2_value(h0), g1 = e4m3x2_value(h1);
              hi[y] = h0 | h1 << 16;
              // (an infinity, which the first term cuts to 448, becomes NaN here)
              lo[y] = e4m3x2(fmaf(f0, 0.0f, f0 - g0.x), fmaf(f1, 0.0f, f1 - g0.y)) |
                      e4m3x2(fmaf(f2, 0.0f, f2 - g1.x), fmaf(f3, 0.0f, f3 - g1.y)) << 16;
            }
            const int ch = half * (D / 32) + x;    // 16-byte chunk of the term's row
            uint8_t *const at = dst + row * 128;
            *reinterpret_cast<uint4 *>(at + ((ch ^ (row & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (D == 128)
              *reinterpret_cast<uint4 *>(at + kQBlockBytes + ((ch ^ (row & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            else
              *reinterpret_cast<uint4 *>(at + (((ch + 4) ^ (row & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_shared();
        warp_arrive(&bars.q_full[qb]);
        return true;
      };
      int nload = 0, tiles = 0;     // of earlier segments
      uint32_t scrubs = 0;
      bool ok = true, more = qwalk.next();
      if (more) {
        ok = split_q();
        more = qwalk.next();
      }
      while (ok && walk.next()) {
        const int nloads = (walk.count + kLoad - 1) / kLoad;
        if (!PAIR && more) {       // the next segment's, while this one runs
          ok = split_q();
          more = ok && qwalk.next();
        }
        for (int jj = (nload ^ team) & 1; ok && jj < nloads; jj += 2) {   // the team's loads: every second one
          const int ld = nload + jj;
          const int sr = ld % C::kRawStages, sl = ld % C::kVStages;
          if (!warp_wait_all(&bars.raw_full[sr], (ld / C::kRawStages) & 1)) {
            ok = false;
            break;
          }
          uint8_t *const src = sraw + sr * C::kRawBytes;
          uint8_t *const dst = sv + sl * C::kLoadBytes;
          if (!SEL) {
            bool special = (walk.tile0 + (jj + 1) * kLoad) * kTile > walk.q.ctx;
#pragma unroll
            for (int x = 0; x < kLoad; ++x) special |= bars.vpage_ok[(tiles + jj * kLoad + x) & 63] == 0u;
            if (special) {
              // V of tokens that some rows do not see has to be finite (0 x NaN is NaN): zero
              // what no row sees, and the NaN codes among the drafted tokens (rows that see
              // them get them back at the end).  128 / kLoad / 64 threads share a key.
              constexpr int kShare = 2 / kLoad, kWords = D / 4 / kShare;
              const int key = t % (kLoad * kTile), part = t / (kLoad * kTile);
              const int pos = (walk.tile0 + jj * kLoad) * kTile + key;
              const int tile = jj * kLoad + key / kTile;
              const bool dead = pos >= walk.q.keys || tile >= walk.count || bars.vpage_ok[(tiles + tile) & 63] == 0u;
              if (dead || pos >= walk.q.ctx) {
#pragma unroll 4
                for (int y = 0; y < kWords; ++y) {
                  uint32_t *const at = reinterpret_cast<uint32_t *>(src + key * D) + part * kWords + (y + t) % kWords;
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
          uint4 v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) v[y] = *reinterpret_cast<const uint4 *>(src + (y * 128 + t) * 16);
          if (!warp_wait_all(&bars.v_empty[sl], ((ld / C::kVStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
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
            mbar_arrive(&bars.v_full[sl]);
            mbar_arrive(&bars.raw_empty[sr]);
          }
        }
        nload += nloads;
        tiles += walk.count;
        if (PAIR && ok && more) {   // one buffer: once this segment's scores are done
          ok = split_q();
          more = ok && qwalk.next();
        }
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

// ---------------------------------------------------------------------------- launch
template <int D, bool F8, bool PAIR, bool SEL>
cudaError_t launch(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm,
                   int num_ctas, cudaStream_t stream) {
  using C = Cfg<D, F8, PAIR, SEL>;
  static std::mutex mu;
  static bool done[128] = {};
  const cudaError_t e = once_per_device(mu, done, [] {
    if (C::kShareRegs) {
      // the register shares come out of what the launch gets: a smaller launch would wait forever
      cudaFuncAttributes f;
      const cudaError_t got = cudaFuncGetAttributes(&f, tree_attention_kernel<D, F8, PAIR, SEL>);
      if (got != cudaSuccess) return got;
      if (f.numRegs != C::kRegsLaunch) return cudaErrorInvalidConfiguration;
    }
    return cudaFuncSetAttribute(tree_attention_kernel<D, F8, PAIR, SEL>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kDynamic);
  });
  if (e != cudaSuccess) return e;
  return launch_cooperative(tree_attention_kernel<D, F8, PAIR, SEL>, num_ctas, C::kThreads, C::kDynamic, stream,
                            qm, km, vm, a);
}

}  // namespace
}  // namespace idx
