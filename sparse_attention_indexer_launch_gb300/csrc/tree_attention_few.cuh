// Attention over a paged cache for at most 64 query vectors per key/value head and item.
//
// So few rows would leave most of a tensor-core tile's M = 128 empty, and re-read them
// from shared memory for every few keys.  Here the keys are M and the rows N:
//
//     S^T = K Q^T   128 keys (two pages) x N rows, TMEM, N = 16, 32 or 64
//     O^T += V^T P^T   D dimensions x N rows, TMEM, with P^T through shared memory
//
// K is operand A as the pages hold it, V^T the MN-major operand A of the same layout
// (64-dimension heads fill M with two readings of the same block).
//
// A softmax thread has one key and all N rows of it.  Every row's probabilities are
// powers of two relative to a reference that the stream's four warps share, set at the
// first tile and raised only when a score passes it by 2^30, so that a tile needs no
// reduction over its keys: each thread checks its own scores, one barrier with an or
// tells the four warps, and only then are the row maxima taken.  Row sums stay with the
// threads until the item ends.  K's scale is one factor per thread, V's another.
//
// Two streams take the even and odd tiles of the CTA's share, each with two S buffers, its
// own O, an MMA-issuing thread and four softmax warps; they are joined in TMEM at the item's
// end.  An item is (request, key/value head, block of tokens) with its tiles in position
// order; the launch's tiles, in item order, are dealt out as one even, contiguous share per
// CTA, and a split item is joined by the CTAs that hold it.
//
// Selected positions: the tiles are 128 entries of a row's selection (then its ancestors),
// and a team of four warps looks them up and copies K, V and scales, 16 bytes a thread.
//
// E4M3 keys feed the tensor core as they are: a row of Q, scaled by a power of two to
// at most 448, is split into two E4M3 terms whose sum it is (exactly, for elements down
// to 2^-9 of the row's largest; to 2^-17 of that below), and S is the sum of both
// terms' products.  P needs bf16's range (two E4M3 terms would drop what lies below
// 2^-18 of the largest, which adds up over a long cache), so V is converted to bf16 in
// shared memory, exactly.
//
// What bounds it.  bf16: memory (4 tokens of 64 heads over 131,072 keys of 8 heads 98 us, 5.5
// TB/s).  E4M3: the chain of a tile's steps in the softmax warps, with the conversion of V
// taking issue slots beside it (the same 84 us, 3.3 TB/s; 64 requests of D = 64 285 us, 2.4
// TB/s): two tiles per step, the tiles' waits hidden behind the TMEM reads and sleeping
// waits were all no faster.  Selected: the copies, at 16 bytes a thread (150 rows over 2,048
// positions of 2 E4M3 heads 103 us); a tile without a single valid entry takes every step all
// the same.  Small calls: the chain launch, lookups, one tile, join (one token over 4,096 keys
// 16.4 us; 8 rows over 2,048 selected positions 22.7 us).
#pragma once

#include "tree_attention_common.cuh"

namespace idx {
namespace {

// Warps 0-3 and 4-7: softmax of streams 0 and 1; 8 and 11: loads of K (and a bf16 Q) and of
// V by TMA; 9 and 10: MMA issuers of streams 0 and 1; from 12 on with an E4M3 cache: the
// split of Q, and V to bf16, in teams of four on a part of every tile; then, for selected
// positions, the team that gathers.
constexpr int kFewKWarp = 8, kFewIssuerWarp = 9, kFewVWarp = 11, kFewConvertWarp = 12;
constexpr int kFewTile = 128;
// Added to the scores of a row without a reference: what any finite score becomes passes kLazy
// and asks for one, and a score of -infinity stays that (added to +infinity it would be NaN).
constexpr float kNoRef = 0x1p127f;

template <int D, bool F8, int N, bool SEL>
struct FewCfg {
  static constexpr int kTileBytes = kFewTile * D * 2;      // K or V of a tile as bf16
  static constexpr int kRawBytes = kFewTile * D;           // ... as E4M3
  static constexpr int kKBytes = F8 ? kRawBytes : kTileBytes;
  static constexpr int kQBytes = N * D * 2;                // bf16, or the two E4M3 terms
  static constexpr int kPBytes = kFewTile * N * 2;         // P^T of a tile
  static constexpr int kPBufs = N == 64 ? 1 : 2;           // per stream
  static constexpr int kQBufs = F8 && N == 64 ? 1 : 2;
  static constexpr int kFixed = kQBufs * kQBytes + 2 * kPBufs * kPBytes;
  // Tiles in flight, as shared memory allows.  The streams take alternate tiles, so the counts
  // are even: a stage then always has the same waiter.  Were they odd, a waiter could come to
  // a stage again before the other's tile in between, and the parity of the barrier would
  // pass for the one that it waits for.
  static constexpr int kKStages = F8 ? (D == 64 ? 6 : N == 16 ? 4 : 2) : D == 64 ? (N == 16 ? 6 : 4) : 2;
  static constexpr int kVStages = F8 ? (D == 64 ? 4 : 2) : D == 64 ? 6 : N == 16 ? 4 : 2;   // as bf16
  static constexpr int kRawStages = F8 ? 4 : 0;                                             // V as E4M3
  static_assert(kKStages % 2 == 0 && kVStages % 2 == 0 && kRawStages % 2 == 0, "one waiter per stage");
  // converting teams of four warps (64 rows leave registers for one), and the team that
  // looks selected positions up
  static constexpr int kTeams = !F8 ? 0 : N < 64 && !SEL ? 2 : 1;
  static constexpr int kLookupWarp = kFewConvertWarp + 4 * kTeams;
  static constexpr int kScaleStages = F8 && D == 64 ? 8 : 4;
  static constexpr int kScaleBytes = F8 && SEL ? kScaleStages * 2 * kFewTile * 4 : 0;
  static constexpr int kThreads = 32 * (kLookupWarp + (SEL ? 4 : 0));
  // Registers per thread after the roles part, where a softmax thread holds a key's scores
  // and row sums; the shares add up to no more than the launch's threads x registers.
  static constexpr bool kShareRegs = kThreads > 384 || N == 64;
  static constexpr int kRegsLaunch = kThreads == 384 ? 168 : kThreads == 512 ? 128 : 96;
  static constexpr int kRegsSoftmax = kThreads == 384 ? 208 : kThreads == 512 ? 176 : N == 16 ? 120 : N == 64 ? 144 : SEL ? 128 : 136;
  static constexpr int kRegsOther = kThreads == 384 ? 88 : kThreads == 512 ? 80 : N == 16 ? 80 : N == 32 && SEL ? 72 : 64;
  static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * kRegsLaunch, "register shares");
  static constexpr int kDynamic = 1024 + kFixed + kKStages * kKBytes + kVStages * kTileBytes + kRawStages * kRawBytes +
                                  kScaleBytes;
};

template <int N>
struct FewBarriers {
  uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8], raw_full[8], raw_empty[8], sc_full[8], sc_empty[8];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2];                    // [stream][S buffer]
  uint64_t p_ready[2][2], pv_done[2][2];    // [stream][P buffer]
  uint64_t o_free[2], drain[2], scrubbed[2];
  // [stream][segment parity]: a stream without tiles in a segment may be one segment ahead
  uint64_t stats[2][2];
  uint32_t tmem_base;
  int abort;
  int32_t two_terms[2][2];         // [stream][P buffer]: a low term follows
  Start found;                     // the share's first request
  Share shares[2];                 // of split items
  int nshare;                      // how many there are
  int warp_sums[20];
  uint32_t pages_ok[32], vpages_ok[32];   // dense: a bit per page of tile k % 32 that was loaded (K, V)
  uint32_t keys_ok[32][4];                // selected: a bit per key of tile k % 32
  int32_t nonfinite[32];                  // segment number + 1 whose drafted tokens' V held NaN or infinity
  alignas(16) float neg_ref[2][N];        // (read four at a time, as q_scale is)
  alignas(16) float q_scale[4][N];        // E4M3: 1 / the row's power of two, [segment % 4]
  float ref[2][N];                        // [stream][row]: the reference (-inf: none yet); neg_ref is what is added to a score
  float keep[2][N];                       // what a raised reference leaves of a row's sums
  float warp_max[2][4][N];
  float row_ref[2][2][N], row_l[2][2][4][N];   // [segment parity][stream], and by warp
  float join[2][3][N];                    // [stream]: factors of both streams' O, 1 / sum
};

// The or of `p` over the 128 threads of a softmax team, which all meet here.
__device__ __forceinline__ bool team_any(int team, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q, r;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "barrier.cta.red.or.pred r, %1, 128, q;\n\tselp.u32 %0, 1, 0, r;\n\t}\n"
      : "=r"(r)
      : "r"(team + 1), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0u;
}
__device__ __forceinline__ void team_sync(int team) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(team + 1) : "memory");
}
__device__ __forceinline__ float warp_max_all(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
// Sums of 32 values over the warp: lane r ends up with value r's.
__device__ __forceinline__ float warp_sums_of(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float mine = up ? v[i + o] : v[i], other = up ? v[i] : v[i + o];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
    }
  return v[0];
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// Copies of this thread arrive on `bar` once they have landed (one of its expected arrivals).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int D, bool F8, int N, bool SEL>
__global__ void __launch_bounds__(FewCfg<D, F8, N, SEL>::kThreads, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const TreeAttnArgs a) {
  using C = FewCfg<D, F8, N, SEL>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ FewBarriers<N> bars;
  uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  uint8_t *const sq = smem;
  uint8_t *const sp = sq + C::kQBufs * C::kQBytes;                 // [stream][buffer]
  uint8_t *const sk = sp + 2 * C::kPBufs * C::kPBytes;
  uint8_t *const sv = sk + C::kKStages * C::kKBytes;
  uint8_t *const sraw = sv + C::kVStages * C::kTileBytes;
  float *const ssc = reinterpret_cast<float *>(sraw + C::kRawStages * C::kRawBytes);   // [stage][K 128, V 128]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const idx_tree_problem &p = a.p;
  const int Hkv = p.cache.Hkv;
  const int G = p.Hq / Hkv;
  const int tb = a.item_tokens;              // tokens of an item, tb * G <= N rows
  constexpr int kBlocks = D / 64;            // 64-dimension blocks of a bf16 operand
  constexpr int kBlockBytes = kFewTile * 128, kQBlockBytes = N * 128;
  constexpr uint32_t kColO = 4 * N;          // S: [stream][buffer] x N columns, then O: [stream] x N

  if (tid < 8) {
    const int s = tid;
    constexpr int loaders = SEL ? 128 : 1;    // selected: each thread of a team with its copies
    mbar_init(&bars.k_full[s], loaders);
    mbar_init(&bars.k_empty[s], 1);
    mbar_init(&bars.v_full[s], F8 ? 4 * C::kTeams : loaders);
    mbar_init(&bars.v_empty[s], 1);
    mbar_init(&bars.raw_full[s], loaders);
    mbar_init(&bars.raw_empty[s], F8 ? 4 * C::kTeams : 1);
    mbar_init(&bars.sc_full[s], 128);
    mbar_init(&bars.sc_empty[s], 4);
    if (s < 2) {
      mbar_init(&bars.q_full[s], F8 ? 4 * C::kTeams : 1);
      mbar_init(&bars.q_empty[s], 2);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars.s_full[s][b], 1);
        mbar_init(&bars.p_ready[s][b], 4);
        mbar_init(&bars.pv_done[s][b], 1);
      }
      mbar_init(&bars.o_free[s], 8);
      mbar_init(&bars.drain[s], 1);
      for (int b = 0; b < 2; ++b) mbar_init(&bars.stats[s][b], 4);
      mbar_init(&bars.scrubbed[s], 4);
    }
    fence_barrier_init();
  }
  if (tid < 32) bars.nonfinite[tid] = 0;
  if (tid == 0) {
    bars.abort = 0;
    bars.nshare = 0;
  }
  if (warp == kFewIssuerWarp) {
    tmem_alloc(&bars.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (!F8) {
    if (tid == kFewKWarp * 32) prefetch_tensormap(&qmap);
    // rows that no token fills stay zero
    for (int x = tid; x < C::kQBufs * C::kQBytes / 16; x += C::kThreads) reinterpret_cast<uint4 *>(sq)[x] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_shared();
  }
  if (!SEL && tid == kFewKWarp * 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
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
  auto give_up = [&]() {
    flag_status(a.status, kStatusTimeout);
    *abort = 1;
  };

  // A wait whose outcome the whole warp shares (so that it leaves its loop together).
  auto warp_wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
    const bool r = mbar_wait(bar, parity, limit, abort);
    if (!r) give_up();
    return __all_sync(0xffffffffu, r);
  };
  auto warp_arrive = [&](uint64_t *bar) {   // one arrival for the warp's threads
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // The copies in flight of `used` loads through a ring of n stages land before the CTA may
  // exit (also after giving up).
  auto land = [&](uint64_t *bar, int n, int used) {
    for (int s = 0; s < n; ++s) {
      if (used <= s) continue;
      const int last = used - 1 - (used - 1 - s) % n;
      if (!mbar_wait(&bar[s], (last / n) & 1, limit, &never)) flag_status(a.status, kStatusTimeout);
    }
  };
  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    // The four warps of a stream meet at hardware barriers, so none may leave alone: a
    // wait that ran out sets `ok`, the warp goes through the motions, and all four leave
    // together at the next team_any.
    if constexpr (C::kShareRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    const int s = warp >> 2, w4 = warp & 3;
    const int key = tid & 127;                                     // key of the tile, and TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(w4) << 21;        // first TMEM lane of the warp << 16
    const uint32_t to = tmem + kColO + s * N + lanes;
    const float c = p.scale * kLog2e;
    float *const neg = bars.neg_ref[s];
    int tiles = 0;      // tiles of earlier segments
    uint32_t n = 0;     // this stream's tiles so far
    uint32_t h = 0;     // and its hand-overs of P
    bool ok = true;
    // the product of hand-over x has completed
    auto settled = [&](uint32_t x) -> bool {
      return warp_wait_all(&bars.pv_done[s][x % C::kPBufs], (x / C::kPBufs) & 1);
    };
    while (walk.next()) {
      const int ctx = walk.q.ctx;
      const int nrow = walk.tokens * G;
      const int row0 = walk.q.row0 + walk.tok0;
      const float *const qs = bars.q_scale[walk.seg & 3];
      if (key < N) {
        bars.ref[s][key] = -INFINITY;
        neg[key] = kNoRef;
      }
      team_sync(s);
      float l[N];
#pragma unroll
      for (int r = 0; r < N; ++r) l[r] = 0.0f;
      const uint32_t h0 = h;
      bool left = false;
      // Dense E4M3: a thread reads its key's two scales itself, a tile of its stream ahead,
      // and the page's id another one ahead.
      const int32_t *const table = p.page_table + static_cast<int64_t>(walk.i) * p.pt_stride + walk.tile0 * 2 + (key >> 6);
      const int table_left = (walk.q.keys + kPage - 1) / kPage - walk.tile0 * 2 - (key >> 6);
      float next_k = 0.0f, next_v = 0.0f;
      int32_t next_page = -1;
      auto page_of = [&](int j) -> int32_t { return j < walk.count && 2 * j < table_left ? table[2 * j] : -1; };
      auto bring_scales = [&](int32_t page) {
        const bool good = page >= 0 && page < p.cache.P;
        const int64_t at = good ? (static_cast<int64_t>(page) * Hkv + walk.head) * kPage + (key & 63) : 0;
        next_k = good ? p.cache.k_scale[at] : 0.0f;
        next_v = good ? p.cache.v_scale[at] : 0.0f;
      };
      if (F8 && !SEL) {
        const int j = (s ^ tiles) & 1;
        bring_scales(page_of(j));
        next_page = page_of(j + 2);
      }
      for (int j = (s ^ tiles) & 1; j < walk.count; j += 2, ++n) {   // the CTA's even or odd tiles
        const int k = tiles + j;
        const int key0 = (walk.tile0 + j) * kFewTile;
        float ck = c, vs = 1.0f;
        if (F8 && !SEL) {
          ck = c * next_k;
          vs = next_v;
          bring_scales(next_page);
          next_page = page_of(j + 4);
        } else if (F8) {
          ok = ok && warp_wait_all(&bars.sc_full[k % C::kScaleStages], (k / C::kScaleStages) & 1);
          ck = c * ssc[(k % C::kScaleStages) * 2 * kFewTile + key];
          vs = ssc[(k % C::kScaleStages) * 2 * kFewTile + kFewTile + key];
          warp_arrive(&bars.sc_empty[k % C::kScaleStages]);
        }
        ok = ok && warp_wait_all(&bars.s_full[s][n & 1], (n >> 1) & 1);
        uint64_t seen = ~0ull;         // rows that see the key
        bool special, open;            // open: every row sees the tile's first key
        if (SEL) {
          const uint32_t *const w = bars.keys_ok[k & 31];
          special = (w[0] & w[1] & w[2] & w[3]) != ~0u;
          open = w[0] & 1u;
          if (!((w[w4] >> lane) & 1u)) seen = 0ull;
        } else {
          const uint32_t pages = bars.pages_ok[k & 31];
          special = key0 + kFewTile > ctx || pages != 3u;
          open = key0 < ctx && (pages & 1u);
          if (special) {
            const int pos = key0 + key;
            if (pos >= walk.q.keys || !((pages >> (key >> 6)) & 1u)) {
              seen = 0ull;
            } else if (pos >= ctx) {
              const int u = pos - ctx;
              seen = 0ull;
#pragma unroll 4
              for (int t = 0; t < walk.tokens; ++t) {
                const bool sees = p.mask != nullptr ? (p.mask[row0 + t] >> u) & 1ull : u <= walk.tok0 + t;
                if (sees) seen |= (G == 64 ? ~0ull : (1ull << G) - 1ull) << (t * G);
              }
            }
          }
        }
        tc_fence_after();
        // Scores relative to the references, in units of log2.  Pass 0 finds whether any
        // passes its reference by too much; if so pass 1 takes the scores themselves, for
        // the rows' maxima, and pass 2 the scores relative to the raised references.
        float e[N];
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          uint32_t x[N];
          __syncwarp();
          const uint32_t ts = tmem + (2 * s + (n & 1)) * N + lanes;
          if constexpr (N == 16) {
            tmem_ld16(ts, x);
          } else {
#pragma unroll
            for (int g = 0; g < N; g += 32) tmem_ld32(ts + g, *reinterpret_cast<uint32_t(*)[32]>(&x[g]));
          }
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < N; ++r) asm volatile("" : "+r"(x[r]));
          if (pass == 0 && h == h0) {
            // the first tile: the references are its first key's scores, where every row sees it.
            // All four warps meet here whether or not: one whose wait ran out may have read `open`
            // from a tile that never came, and none may be left at a barrier alone.
            if (open && key == 0) {
#pragma unroll
              for (int r = 0; r < N; ++r) {
                const float m = __uint_as_float(x[r]) * ck * (F8 ? qs[r] : 1.0f);
                const bool fine = m - m == 0.0f;    // else the row's maximum is taken below (kNoRef asks for it)
                bars.ref[s][r] = fine ? m : -INFINITY;
                neg[r] = fine ? -m : kNoRef;
              }
            }
            team_sync(s);
          }
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int r = 0; r < N; r += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(neg + r);
            float2 e0, e1;
            const float2 x0 = make_float2(__uint_as_float(x[r]), __uint_as_float(x[r + 1]));
            const float2 x1 = make_float2(__uint_as_float(x[r + 2]), __uint_as_float(x[r + 3]));
            const float2 cc = make_float2(ck, ck);
            if (F8) {
              const float4 q = *reinterpret_cast<const float4 *>(qs + r);
              e0 = __ffma2_rn(__fmul2_rn(x0, cc), make_float2(q.x, q.y), make_float2(m.x, m.y));
              e1 = __ffma2_rn(__fmul2_rn(x1, cc), make_float2(q.z, q.w), make_float2(m.z, m.w));
            } else {
              e0 = __ffma2_rn(x0, cc, make_float2(m.x, m.y));
              e1 = __ffma2_rn(x1, cc, make_float2(m.z, m.w));
            }
            e[r] = e0.x;
            e[r + 1] = e0.y;
            e[r + 2] = e1.x;
            e[r + 3] = e1.y;
          }
          if (special) {
#pragma unroll
            for (int r = 0; r < N; ++r)
              if (!((static_cast<uint32_t>(seen >> (r & 32)) >> (r & 31)) & 1u)) e[r] = -INFINITY;
          }
          if (pass == 2) break;
          if (pass == 0) {
#pragma unroll
            for (int r = 0; r < N; r += 8)
#pragma unroll
              for (int z = 0; z < 4; ++z) t4[z] = max3(t4[z], e[r + 2 * z], e[r + 2 * z + 1]);
            const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
            if (!team_any(s, !ok || top > kLazy)) break;
            if (team_any(s, !ok)) {
              left = true;
              break;
            }
            if (key < N) neg[key] = 0.0f;
            team_sync(s);
            continue;
          }
          // the rows' maxima over the keys, and the references that they raise
          float mine[(N + 31) / 32] = {};
#pragma unroll
          for (int r = 0; r < N; ++r) {
            const float m = warp_max_all(e[r]);
            if (lane == (r & 31)) mine[r >> 5] = m;
          }
#pragma unroll
          for (int g = 0; g < (N + 31) / 32; ++g)
            if (lane + 32 * g < N) bars.warp_max[s][w4][lane + 32 * g] = mine[g];
          team_sync(s);
          if (key < N) {
            const float m = fmaxf(fmaxf(bars.warp_max[s][0][key], bars.warp_max[s][1][key]),
                                  fmaxf(bars.warp_max[s][2][key], bars.warp_max[s][3][key]));
            const float old = bars.ref[s][key];
            const float now = m > old + kLazy || old == -INFINITY ? fmaxf(m, old) : old;
            bars.ref[s][key] = now;
            neg[key] = now == -INFINITY ? kNoRef : -now;
            bars.keep[s][key] = old == -INFINITY ? 0.0f : ex2(old - now);
          }
          team_sync(s);
#pragma unroll
          for (int r = 0; r < N; ++r) l[r] *= bars.keep[s][r];
          if (h != h0) {
            // O once the products before have completed (the last two may be under way)
            if (C::kPBufs > 1 && h - h0 > 1) ok = ok && settled(h - 2);
            ok = ok && settled(h - 1);
            tc_fence_after();
            __syncwarp();
            if (ok) {
#pragma unroll 1
              for (int g = 0; g < N; g += 8) {
                uint32_t o[8];
                tmem_ld8(to + g, o);
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < 8; ++r) asm volatile("" : "+r"(o[r]));
#pragma unroll
                for (int r = 0; r < 8; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * bars.keep[s][g + r]);
                tmem_st8(to + g, o);
              }
              tmem_wait_st();
            }
            tc_fence_before();
          }
        }
        if (left) break;
        // V of tokens that some rows do not see has to be finite (0 x NaN is NaN): zero
        // what no row sees, and what is not finite among the drafted tokens (rows that
        // see it get it back at the end)
        if (!SEL && !F8 && special) {
          const int sl = k % C::kVStages;
          // (the stream's product before first: with two stages its V stood in the same one, and
          // while that had not come this wait's parity would pass for it)
          if (h != h0) ok = ok && settled(h - 1);
          ok = ok && warp_wait_all(&bars.v_full[sl], (k / C::kVStages) & 1);
          const int pos = key0 + key;
          const bool dead = pos >= walk.q.keys || !((bars.pages_ok[k & 31] >> (key >> 6)) & 1u);
          if (ok && (dead || pos >= ctx)) {
            auto chunk = [&](int y) -> uint4 * {
              return reinterpret_cast<uint4 *>(sv + sl * C::kTileBytes + (y >> 3) * kBlockBytes + key * 128 +
                                               ((y + key) & 7) * 16);
            };
            bool bad = false;
            if (!dead) {   // 0 x a value is NaN where it is not finite
              __nv_bfloat162 z = __float2bfloat162_rn(0.0f);
#pragma unroll 4
              for (int y = 0; y < kBlocks * 8; ++y) {
                const uint4 v = *chunk(y);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  z = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(w[x]), __float2bfloat162_rn(0.0f), z);
              }
              bad = __hisnan(__low2bfloat16(z)) || __hisnan(__high2bfloat16(z));
            }
            if (dead || bad) {
#pragma unroll 1
              for (int y = 0; y < kBlocks * 8; ++y) {
                uint4 *const at = chunk(y);
                uint32_t w[4] = {};
                if (bad) {
                  const uint4 v = *at;
                  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    if ((w[x] & 0x7F80u) == 0x7F80u) w[x] &= 0xFFFF0000u;
                    if ((w[x] & 0x7F800000u) == 0x7F800000u) w[x] &= 0xFFFFu;
                  }
                }
                *at = make_uint4(w[0], w[1], w[2], w[3]);
              }
              if (bad) bars.nonfinite[walk.seg & 31] = walk.seg + 1;
            }
          }
          __syncwarp();
        }
        // P.  It is rounded to bf16 for the product with V.  That leaves an error nearly as
        // large as the output's own rounding (relative to the output 0.9e-3 over 128 keys to
        // 1.5e-3 over 65,536, beside 1.7e-3), for half the products that two terms would take.
        // The few visible keys of a special tile average out less (up to 2^-8 of one value):
        // there a second hand-over brings what the rounding left.
#pragma unroll
        for (int r = 0; r < N; r += 2) {
          const float2 y = make_float2(ex2(e[r]), ex2(e[r + 1]));
          const float2 sum = __fadd2_rn(make_float2(l[r], l[r + 1]), y);
          l[r] = sum.x;
          l[r + 1] = sum.y;
          const float2 z = F8 ? __fmul2_rn(y, make_float2(vs, vs)) : y;
          e[r] = z.x;
          e[r + 1] = z.y;
        }
        if (F8 && special) {   // a stale scale may be NaN
#pragma unroll
          for (int r = 0; r < N; ++r)
            if (!((static_cast<uint32_t>(seen >> (r & 32)) >> (r & 31)) & 1u)) e[r] = 0.0f;
        }
#pragma unroll 1
        for (int more = special; more >= 0; --more) {
          // the buffer's product before has to have completed
          if (h - h0 >= C::kPBufs) ok = ok && settled(h - C::kPBufs);
          uint8_t *const row = sp + (s * C::kPBufs + h % C::kPBufs) * C::kPBytes + key * (2 * N);
#pragma unroll
          for (int r = 0; r < N; r += 8) {
            uint32_t w[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) w[z] = pack_bf16(e[r + 2 * z], e[r + 2 * z + 1]);
            const int sw = N == 64 ? key & 7 : N == 32 ? (key >> 1) & 3 : (key >> 2) & 1;
            *reinterpret_cast<uint4 *>(row + (((r >> 3) ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (key == 0) bars.two_terms[s][h % C::kPBufs] = more;
          fence_proxy_async_shared();
          tc_fence_before();
          warp_arrive(&bars.p_ready[s][h % C::kPBufs]);
          ++h;
          if (more) {   // what the rounding left (an infinity, of a scale, leaves nothing)
#pragma unroll
            for (int r = 0; r < N; ++r) {
              const float rest = e[r] - __bfloat162float(__float2bfloat16_rn(e[r]));
              e[r] = rest == rest ? rest : 0.0f;
            }
          }
        }
      }
      if (left) break;

      // -------------------------------------------------------------- end of the segment
      if (C::kPBufs > 1 && h - h0 > 1) ok = ok && settled(h - 2);
      if (h != h0) ok = ok && settled(h - 1);
      const int sp2 = walk.seg & 1;
#pragma unroll
      for (int g = 0; g < N; g += 32) {
        float v[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) v[r] = g + r < N ? l[g + r] : 0.0f;
        const float sum = warp_sums_of(v, lane);
        if (g + lane < N) bars.row_l[sp2][s][w4][g + lane] = sum;
      }
      if (key < N) bars.row_ref[sp2][s][key] = bars.ref[s][key];
      tc_fence_before();
      warp_arrive(&bars.stats[s][sp2]);
      ok = ok && warp_wait_all(&bars.stats[0][sp2], (walk.seg >> 1) & 1) && warp_wait_all(&bars.stats[1][sp2], (walk.seg >> 1) & 1);
      tc_fence_after();
      const int slot = (walk.first ? 0 : 1) + 2 * static_cast<int>(blockIdx.x);
      if (key < N) {
        float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          l0 += bars.row_l[sp2][0][w][key];
          l1 += bars.row_l[sp2][1][w][key];
        }
        float m0 = bars.row_ref[sp2][0][key], m1 = bars.row_ref[sp2][1][key];
        // a NaN among the visible scores takes the whole row, in every join
        if (l0 != l0) m0 = INFINITY;
        if (l1 != l1) m1 = INFINITY;
        const float m = fmaxf(m0, m1);
        const float f0 = m0 == -INFINITY ? 0.0f : ex2(m0 - m), f1 = m1 == -INFINITY ? 0.0f : ex2(m1 - m);
        const float sum = l0 * f0 + l1 * f1;
        bars.join[s][0][key] = f0;
        bars.join[s][1][key] = f1;
        bars.join[s][2][key] = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (s == 0 && key < nrow && ok) {
          if (!walk.whole) {
            a.part_ml[static_cast<int64_t>(slot) * 128 + key] = make_float2(m, sum);
          } else if (a.lse != nullptr) {
            a.lse[static_cast<int64_t>(row0 + key / G) * p.Hq + walk.head * G + key % G] =
                sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
          }
        }
      }
      team_sync(s);
      // O^T: a lane per dimension.  Each team writes half of the rows; with 64 dimensions
      // lanes 64-127 hold the same as 0-63 and take every second group of four rows.
      const bool poison = *reinterpret_cast<volatile int32_t *>(&bars.nonfinite[walk.seg & 31]) == walk.seg + 1;
      const int d = D == 128 ? key : key & 63;
      const uint32_t o0 = tmem + kColO + lanes;
      const int odd = tiles & 1;      // (of the segment's first tile)
      const bool has0 = odd < walk.count, has1 = (odd ^ 1) < walk.count;   // the streams that had tiles
      // an item's rows are G heads of consecutive tokens
      uint16_t *const out = a.out + (static_cast<int64_t>(row0) * p.Hq + walk.head * G) * D + d;
      float *const part = a.part_o + share_at<D, false>(slot, 128, 0, d);
      auto put = [&](int row, float o) {
        if (!walk.whole) {
          part[row * D] = o;
        } else {
          const int tok = row / G;
          out[static_cast<int64_t>(tok * p.Hq + row - tok * G) * D] = static_cast<uint16_t>(pack_bf16(o * bars.join[s][2][row], 0.0f));
        }
      };
#pragma unroll 1
      for (int g = s * (N / 2); g < (s + 1) * (N / 2); g += 8) {
        if (g >= nrow) break;
        uint32_t x0[8], x1[8];
        __syncwarp();
        if (has0) tmem_ld8(o0 + g, x0);
        if (has1) tmem_ld8(o0 + N + g, x1);
        tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          asm volatile("" : "+r"(x0[r]));
          asm volatile("" : "+r"(x1[r]));
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (D == 64 && ((r >> 2) != (key >> 6))) continue;
          const int row = g + r;
          if (row >= nrow || !ok) continue;
          const float f0 = bars.join[s][0][row], f1 = bars.join[s][1][row];
          float o = has0 ? __uint_as_float(x0[r]) * f0 : 0.0f;
          if (has1) o += __uint_as_float(x1[r]) * f1;
          if (bars.join[s][2][row] == 0.0f) o = 0.0f;
          if (!poison) {
            put(row, o);
            continue;
          }
          const int tok = row / G;
          {   // what was zeroed for the rows that do not see it
            const int t = walk.tok0 + tok;
            const uint64_t mask = p.mask != nullptr ? p.mask[row0 + tok] : (2ull << t) - 1ull;
            for (int u = 0; u < walk.q.tokens; ++u) {
              const int pos = ctx + u;
              if (!((mask >> u) & 1ull) || pos >= walk.q.keys || pos < walk.tile0 * kFewTile ||
                  pos >= (walk.tile0 + walk.count) * kFewTile)
                continue;
              const int32_t pg = p.page_table[static_cast<int64_t>(walk.i) * p.pt_stride + pos / kPage];
              if (pg < 0 || pg >= p.cache.P) continue;
              const int64_t at = pg * p.cache.page_stride + (pos % kPage) * p.cache.token_stride +
                                 walk.head * p.cache.head_stride + d;
              float v;
              if (F8) v = static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(p.cache.v)[at]);
              else v = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.cache.v)[at]);
              if (!isfinite(v)) o += v;
            }
          }
          put(row, o);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.o_free[0]);
        mbar_arrive(&bars.o_free[1]);
      }
      tiles += walk.count;
      if (!walk.whole && tid == 0) bars.shares[bars.nshare++] = share_of(walk, share, G);
    }
    if (!ok) give_up();
    join_items<D, false>(a, bars.shares, &bars.nshare, ok);
  } else if (warp < kFewConvertWarp) {
    if constexpr (C::kShareRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kFewKWarp || (!SEL && warp == kFewVWarp)) {
      // -------------------------------------------------------------- loads
      // K's warp also brings a bf16 Q.  Selected positions are
      // brought by a team of their own.
      const bool is_v = warp == kFewVWarp;
      const int stages = is_v ? (F8 ? C::kRawStages : C::kVStages) : C::kKStages;
      constexpr int kBytes = C::kKBytes;       // of a load: E4M3 or bf16, K or V
      uint64_t *const full = is_v ? (F8 ? bars.raw_full : bars.v_full) : bars.k_full;
      uint64_t *const empty = is_v ? (F8 ? bars.raw_empty : bars.v_empty) : bars.k_empty;
      uint8_t *const ring = is_v ? (F8 ? sraw : sv) : sk;
      int stage = 0;          // of the next load
      uint32_t phase = 1;     // its empty barrier's
      int nload = 0;          // loads (tiles) so far
      int nq = 0;             // Q loads so far
      bool ok = true;
      auto warp_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        int r = 1;
        if (lane == 0) r = mbar_wait(bar, parity, limit, abort);
        return __shfl_sync(0xffffffffu, r, 0) != 0;
      };
      while (ok && walk.next()) {
        if (!F8 && !is_v) {
          const int qb = walk.seg % C::kQBufs;
          if (!warp_wait(&bars.q_empty[qb], ((walk.seg / C::kQBufs) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars.q_full[qb], static_cast<uint32_t>(kBlocks * G * tb * 128));
            for (int b = 0; b < kBlocks; ++b)
              tma_load_3d(sq + qb * C::kQBytes + b * kQBlockBytes, &qmap, b * 64, walk.head * G,
                          walk.q.row0 + walk.tok0, &bars.q_full[qb]);
          }
          ++nq;
        }
        const int32_t *const table = p.page_table + static_cast<int64_t>(walk.i) * p.pt_stride;
        if constexpr (!SEL) {
          // ---------------------------------------------------------- pages by TMA
          const void *const map = is_v ? &vmap : &kmap;
          uint32_t *const oks = is_v ? bars.vpages_ok : bars.pages_ok;
          const int npages = (walk.q.keys + kPage - 1) / kPage;
          // One thread, without a step that it would share with its warp: at a few hundred
          // cycles per tile it is close to the kernel's pace.  Page ids are read three tiles
          // ahead (-2: past the request's pages).
          if (lane == 0) {
            auto fetch = [&](int j) -> int2 {
              const int pg = (walk.tile0 + j) * 2;
              const int2 ids = make_int2(-2, -2);
              return j >= walk.count ? ids
                                     : make_int2(pg < npages ? table[pg] : -2, pg + 1 < npages ? table[pg + 1] : -2);
            };
            int2 next[3] = {fetch(0), fetch(1), fetch(2)};
            for (int j = 0; j < walk.count; ++j) {
              const int32_t pg[2] = {next[0].x, next[0].y};
              next[0] = next[1];
              next[1] = next[2];
              next[2] = fetch(j + 3);
              uint32_t good = 0;
#pragma unroll
              for (int x = 0; x < 2; ++x) good |= static_cast<uint32_t>(pg[x] >= 0 && pg[x] < p.cache.P) << x;
              if (!mbar_wait(&empty[stage], phase, limit, abort)) {
                ok = false;
                break;
              }
              uint8_t *const dst = ring + stage * kBytes;
              oks[nload & 31] = good;
              if ((!(good & 1u) && pg[0] != -2) || (!(good & 2u) && pg[1] != -2)) flag_status(a.status, kStatusBadPage);
              mbar_arrive_expect_tx(&full[stage], __popc(good) * static_cast<uint32_t>(kBytes / 2));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                if (!((good >> x) & 1u)) continue;
                if constexpr (F8) {
                  tma_load_4d(dst + x * (kPage * D), map, 0, 0, walk.head, pg[x], &full[stage]);
                } else {
#pragma unroll
                  for (int b = 0; b < kBlocks; ++b)
                    tma_load_4d(dst + b * kBlockBytes + x * (kPage * 128), map, b * 64, 0, walk.head, pg[x], &full[stage]);
                }
              }
              ++nload;
              if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
      if (!ok && lane == 0) give_up();
      if (lane == 0) {
        land(bars.q_full, C::kQBufs, nq);
        land(full, stages, nload);
      }
    } else if (warp != kFewVWarp && lane == 0) {
      // -------------------------------------------------------------- MMA issuers
      // Per stream: S of two tiles; then, tile by tile, O += P V for each term of its P, and
      // S of the second next tile (the S it replaces has been read: its P is there).
      const int s = warp - kFewIssuerWarp;
      const uint32_t to = tmem + kColO + s * N;
      constexpr uint32_t kAMn = 1u << 15;
      const uint32_t idesc_s = umma_idesc(F8 ? 0u : 1u, N), idesc_o = umma_idesc(1u, N) | kAMn | kIdescBMn;
      // P^T: keys' rows of N values in the swizzle of their size
      constexpr uint64_t kPSwizzle = N == 64 ? 2 : N == 32 ? 4 : 6;
      int tiles = 0;      // tiles of earlier segments
      uint32_t ns = 0;    // this stream's S so far
      uint32_t h = 0;     // hand-overs of P so far
      bool ok = true, any = false;
      while (ok && walk.next()) {
        const int qb = walk.seg % C::kQBufs;
        if (!mbar_wait(&bars.q_full[qb], (walk.seg / C::kQBufs) & 1, limit, abort)) {
          ok = false;
          break;
        }
        const int j0 = (s ^ tiles) & 1;      // the stream's first tile
        if (j0 >= walk.count) mbar_arrive(&bars.q_empty[qb]);
        const uint32_t qaddr = smem_u32(sq + qb * C::kQBytes);
        auto scores = [&](int j) -> bool {   // S of tile j
          const int k = tiles + j, sl = k % C::kKStages;
          if (!mbar_wait(&bars.k_full[sl], (k / C::kKStages) & 1, limit, abort)) return false;
          if (SEL) fence_proxy_async_shared();   // the gatherers' copies
          tc_fence_after();
          const uint32_t d = tmem + (2 * s + (ns & 1)) * N;
          const uint32_t kaddr = smem_u32(sk + sl * C::kKBytes);
          if constexpr (F8) {
            // both terms of Q over the same keys: D = 128: 128-byte rows, the terms a block
            // apart; D = 64: the terms side by side in 128-byte rows, keys in 64-byte rows
            const uint64_t kdesc = D == 128 ? umma_desc_sw128(kaddr) : umma_desc_sw64(kaddr);
            const uint64_t qdesc = umma_desc_sw128(qaddr);
#pragma unroll
            for (int kk = 0; kk < 2 * D / 32; ++kk) {
              const int term = kk / (D / 32), x = kk % (D / 32);
              umma_f8(d, kdesc + ((x * 32) >> 4), qdesc + ((term * (D == 128 ? kQBlockBytes : 64) + x * 32) >> 4), idesc_s,
                      kk > 0);
            }
          } else {
            const uint64_t kdesc = umma_desc_sw128(kaddr), qdesc = umma_desc_sw128(qaddr);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_f16(d, kdesc + (((kk >> 2) * kBlockBytes + (kk & 3) * 32) >> 4),
                       qdesc + (((kk >> 2) * kQBlockBytes + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
          }
          umma_commit(&bars.s_full[s][ns & 1]);
          umma_commit(&bars.k_empty[sl]);
          if (j + 2 >= walk.count) umma_commit(&bars.q_empty[qb]);
          any = true;
          ++ns;
          return true;
        };
        for (int j = j0; ok && j < walk.count && j < j0 + 4; j += 2) ok = scores(j);
        for (int j = j0; ok && j < walk.count; j += 2) {
          const int k = tiles + j, sl = k % C::kVStages;
          bool more = true;
          for (int term = 0; more; ++term) {
            const int pb = h % C::kPBufs;
            if (!mbar_wait(&bars.p_ready[s][pb], (h / C::kPBufs) & 1, limit, abort) ||
                (term == 0 && j == j0 && !mbar_wait(&bars.o_free[s], (walk.seg & 1) ^ 1, limit, abort)) ||
                (term == 0 && !mbar_wait(&bars.v_full[sl], (k / C::kVStages) & 1, limit, abort))) {
              ok = false;
              break;
            }
            if (SEL && !F8 && term == 0) fence_proxy_async_shared();
            tc_fence_after();
            more = *reinterpret_cast<volatile int32_t *>(&bars.two_terms[s][pb]) != 0;
            const uint32_t vaddr = smem_u32(sv + sl * C::kTileBytes);
            const uint32_t paddr = smem_u32(sp + (s * C::kPBufs + pb) * C::kPBytes);
            // D = 64: the second 64 of M read the same block again
            const uint64_t vdesc = umma_desc_mn(vaddr, D == 128 ? kBlockBytes : 0);
            uint64_t pdesc = static_cast<uint64_t>((paddr >> 4) & 0x3FFFu);
            pdesc |= static_cast<uint64_t>(1u) << 16;
            pdesc |= static_cast<uint64_t>((8 * 2 * N) >> 4) << 32;     // the next eight keys
            pdesc |= static_cast<uint64_t>(1u) << 46;
            pdesc |= kPSwizzle << 61;
#pragma unroll
            for (int kk = 0; kk < kFewTile / 16; ++kk)
              umma_f16(to, vdesc + ((kk * 16 * 128) >> 4), pdesc + ((kk * 16 * 2 * N) >> 4), idesc_o,
                       j > j0 || term > 0 || kk > 0);
            umma_commit(&bars.pv_done[s][pb]);
            ++h;
          }
          if (!ok) break;
          umma_commit(&bars.v_empty[sl]);
          if (j + 4 < walk.count) ok = scores(j + 4);
        }
        tiles += walk.count;
      }
      if (!ok) {
        give_up();
        if (any) {   // MMAs in flight read shared memory and TMEM: wait for them
          umma_commit(&bars.drain[s]);
          if (!mbar_wait(&bars.drain[s], 0, limit, &never)) flag_status(a.status, kStatusTimeout);
        }
      }
    }
  } else if (SEL && warp >= C::kLookupWarp) {
    if constexpr (SEL) {
      // -------------------------------------------------------------- selected positions
      // A thread looks one key of every tile up: its entry of the selection, the page, the
      // slot.  Each step's load is issued a tile ahead of the next step.  A warp then brings
      // its 32 keys' K, V and scales.
      if constexpr (C::kShareRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
      const int key = tid - C::kLookupWarp * 32, w4 = key >> 5;
      constexpr int kVRing = F8 ? C::kRawStages : C::kVStages;
      uint64_t *const vfull = F8 ? bars.raw_full : bars.v_full;
      int k = 0;     // tiles so far
      bool ok = true;
      while (ok && walk.next()) {
        const int32_t *const table = p.page_table + static_cast<int64_t>(walk.i) * p.pt_stride;
        const int r = walk.q.row0 + walk.tok0;
        const uint64_t mask = p.mask != nullptr ? p.mask[r] : (2ull << walk.tok0) - 1ull;
        const int32_t *const sel = a.sel + static_cast<int64_t>(r) * a.sel_k;
        int n = walk.tile0 * kFewTile + key;
        const int nend = (walk.tile0 + walk.count) * kFewTile;
        auto entry = [&](int m) -> int32_t { return m < nend && m < a.sel_k ? sel[m] : -1; };
        auto position = [&](int m, int32_t e) -> int32_t {   // logical position, -1 for none
          if (m < a.sel_k) return e >= 0 && e < walk.q.ctx ? e : -1;
          const int u = m - a.sel_k;
          return u < walk.q.tokens && ((mask >> u) & 1ull) && walk.q.ctx + u < walk.q.keys ? walk.q.ctx + u : -1;
        };
        int32_t pos = position(n, entry(n));
        int32_t page = pos >= 0 ? table[pos / kPage] : -1;
        int32_t e = entry(n + kFewTile);
        for (; n < nend; n += kFewTile, ++k) {
          int32_t slot = -1;           // page * 64 + token
          if (pos >= 0) {
            if (page >= 0 && page < p.cache.P) slot = page * kPage + pos % kPage;
            else flag_status(a.status, kStatusBadPage);
          }
          pos = n + kFewTile < nend ? position(n + kFewTile, e) : -1;
          page = pos >= 0 ? table[pos / kPage] : -1;
          e = entry(n + 2 * kFewTile);
          const uint32_t bits = __ballot_sync(0xffffffffu, slot >= 0);
          const int ks = k % C::kKStages, vs = k % kVRing, ss = k % C::kScaleStages;
          if (!warp_wait_all(&bars.k_empty[ks], ((k / C::kKStages) & 1) ^ 1) ||
              (F8 && !warp_wait_all(&bars.sc_empty[ss], ((k / C::kScaleStages) & 1) ^ 1))) {
            ok = false;
            break;
          }
          if (lane == 0) bars.keys_ok[k & 31][w4] = bits;
          if constexpr (F8) {
            const int64_t at = slot < 0 ? 0 : (static_cast<int64_t>(slot / kPage) * Hkv + walk.head) * kPage + slot % kPage;
            const uint32_t to = smem_u32(ssc + ss * 2 * kFewTile + key);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(p.cache.k_scale + at), "r"(slot < 0 ? 0 : 4)
                         : "memory");
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + kFewTile * 4), "l"(p.cache.v_scale + at),
                         "r"(slot < 0 ? 0 : 4)
                         : "memory");
            cp_async_arrive(&bars.sc_full[ss]);
          }
          // K first, then V once its stage is free: S runs up to four tiles ahead of the
          // products that free V's stages, and must not wait for them.
          const int64_t off = slot < 0 ? -1
                                       : (slot / kPage * p.cache.page_stride + slot % kPage * p.cache.token_stride +
                                          walk.head * p.cache.head_stride) *
                                             (F8 ? 1 : 2);
#pragma unroll
          for (int is_v = 0; is_v < 2; ++is_v) {
            if (is_v && !warp_wait_all(&(F8 ? bars.raw_empty : bars.v_empty)[vs], ((k / kVRing) & 1) ^ 1)) {
              ok = false;
              break;
            }
            uint8_t *const dst = is_v ? (F8 ? sraw : sv) + vs * C::kKBytes : sk + ks * C::kKBytes;
            // 16 bytes per thread: D / 16 or D / 8 lanes bring one key
            constexpr int kLanes = F8 ? D / 16 : D / 8, kKeysAtOnce = 32 / kLanes;
            const int ch = lane % kLanes;
#pragma unroll 8
            for (int y = 0; y < kLanes; ++y) {
              const int from = y * kKeysAtOnce + lane / kLanes, at_key = w4 * 32 + from;
              const int64_t o = __shfl_sync(0xffffffffu, off, from);
              uint32_t at;   // bf16: blocks of 128-byte rows, swizzled; E4M3 K: rows of D, swizzled; V: rows of D
              if (!F8) at = (ch >> 3) * kBlockBytes + at_key * 128 + (((ch & 7) ^ (at_key & 7)) << 4);
              else if (is_v) at = at_key * D + ch * 16;
              else at = at_key * D + ((D == 128 ? ch ^ (at_key & 7) : ch ^ ((at_key >> 1) & 3)) << 4);
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + at)),
                           "l"(static_cast<const uint8_t *>(is_v ? p.cache.v : p.cache.k) + (o < 0 ? 0 : o) + ch * 16),
                           "r"(o < 0 ? 0 : 16)
                           : "memory");
            }
            cp_async_arrive(is_v ? &vfull[vs] : &bars.k_full[ks]);
          }
          if (!ok) break;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok && lane == 0) give_up();
    }
  } else {
    if constexpr (F8) {
      // -------------------------------------------------------------- E4M3: Q split, V to bf16
      if constexpr (C::kShareRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
      const int team = (warp - kFewConvertWarp) >> 2, t = (tid - kFewConvertWarp * 32) & 127;
      Walk qwalk(a, t0, t1, first.req, first.base, first.q);     // the segment whose Q is next
      // Q of qwalk's segment: D / 16 lanes per row with 16 elements each; rows without a
      // token are zero.
      auto split_q = [&]() -> bool {
        const int qb = qwalk.seg % C::kQBufs;
        if (!warp_wait_all(&bars.q_empty[qb], ((qwalk.seg / C::kQBufs) & 1) ^ 1)) return false;
        constexpr int kLanes = D / 16;
        const int nrow = qwalk.tokens * G;
        for (int id = tid - kFewConvertWarp * 32; id < N * kLanes; id += 128 * C::kTeams) {
          const int row = id / kLanes, ch = id % kLanes;
          uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
          if (row < nrow) {
            const uint4 *const src = reinterpret_cast<const uint4 *>(
                static_cast<const uint16_t *>(p.q) +
                static_cast<int64_t>(qwalk.q.row0 + qwalk.tok0 + row / G) * p.q_row_stride +
                static_cast<int64_t>(qwalk.head * G + row % G) * D + ch * 16);
            v[0] = __ldg(src);
            v[1] = __ldg(src + 1);
          }
          const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
          // the row's largest exponent (of the finite elements: NaN and infinity stay what they are)
          uint32_t top = 0;
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const uint32_t lo = w[y] & 0x7FFFu, hi = (w[y] >> 16) & 0x7FFFu;
            if (lo < 0x7F80u) top = max(top, lo);
            if (hi < 0x7F80u) top = max(top, hi);
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          // 2^e takes it to (224, 448]; rows below 2^-112 stop at 2^120
          const int e = min(((top & 0x7Fu) <= 0x60u ? 8 : 7) - (static_cast<int>(top >> 7) - 127), 120);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          if (ch == 0) bars.q_scale[qwalk.seg & 3][row] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float f0 = __uint_as_float(w[2 * y] << 16) * up, f1 = __uint_as_float(w[2 * y] & 0xFFFF0000u) * up;
            const float f2 = __uint_as_float(w[2 * y + 1] << 16) * up, f3 = __uint_as_float(w[2 * y + 1] & 0xFFFF0000u) * up;
            const uint32_t h0 = e4m3x2(f0, f1), h1 = e4m3x2(f2, f3);
            const float2 g0 = e4m3x2_value(h0), g1 = e4m3x2_value(h1);
            hi[y] = h0 | h1 << 16;
            // (an infinity, which the first term cuts to 448, becomes NaN here)
            lo[y] = e4m3x2(fmaf(f0, 0.0f, f0 - g0.x), fmaf(f1, 0.0f, f1 - g0.y)) |
                    e4m3x2(fmaf(f2, 0.0f, f2 - g1.x), fmaf(f3, 0.0f, f3 - g1.y)) << 16;
          }
          uint8_t *const at = sq + qb * C::kQBytes + row * 128;
          *reinterpret_cast<uint4 *>(at + ((ch ^ (row & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if constexpr (D == 128)
            *reinterpret_cast<uint4 *>(at + kQBlockBytes + ((ch ^ (row & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          else
            *reinterpret_cast<uint4 *>(at + (((ch + 4) ^ (row & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_shared();
        warp_arrive(&bars.q_full[qb]);
        return true;
      };
      int tiles = 0;     // of earlier segments
      uint32_t scrubs = 0;
      bool ok = true, more = qwalk.next();
      if (more) {
        ok = split_q();
        more = qwalk.next();
      }
      while (ok && walk.next()) {
        if (C::kQBufs > 1 && more) {       // the next segment's, while this one runs
          ok = split_q();
          more = ok && qwalk.next();
        }
        for (int j = 0; j < walk.count; ++j) {   // each team a half of every tile
          const int k = tiles + j;
          const int sr = k % C::kRawStages, sl = k % C::kVStages;
          if (!warp_wait_all(&bars.raw_full[sr], (k / C::kRawStages) & 1)) {
            ok = false;
            break;
          }
          constexpr int kKeys = kFewTile / C::kTeams;      // of a team
          uint8_t *const src = sraw + sr * C::kRawBytes + team * kKeys * D;
          uint8_t *const dst = sv + sl * C::kTileBytes + team * kKeys * 128;
          if (!SEL) {
            const int key0 = (walk.tile0 + j) * kFewTile;
            const uint32_t pages = bars.vpages_ok[k & 31];
            if (key0 + kFewTile > walk.q.ctx || pages != 3u) {
              // V of tokens that some rows do not see has to be finite (0 x NaN is NaN): zero
              // what no row sees, and the NaN codes among the drafted tokens (rows that see
              // them get them back at the end).  One or two threads per key.
              constexpr int kShare = 128 / kKeys, kWords = D / 4 / kShare;
              const int key = t % kKeys, at_key = team * kKeys + key, pos = key0 + at_key;
              const bool dead = pos >= walk.q.keys || !((pages >> (at_key >> 6)) & 1u);
              if (dead || pos >= walk.q.ctx) {
#pragma unroll 4
                for (int y = 0; y < kWords; ++y) {
                  uint32_t *const at =
                      reinterpret_cast<uint32_t *>(src + key * D) + (t / kKeys) * kWords + (y + t) % kWords;
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
          constexpr int kChunks = D / 16;                   // 16-byte chunks of codes per key
          constexpr int kMine = kKeys * kChunks / 128;      // a thread's chunks
          constexpr int kBatch = kMine < 4 ? kMine : 4;
          uint4 v[kBatch];
#pragma unroll
          for (int y = 0; y < kBatch; ++y) v[y] = *reinterpret_cast<const uint4 *>(src + (y * 128 + t) * 16);
          if (!warp_wait_all(&bars.v_empty[sl], ((k / C::kVStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int y = 0; y < kMine; ++y) {
            const int key = (y * 128 + t) / kChunks, ch = t % kChunks;
            uint4 &w = v[y % kBatch];
            const uint2 a0 = e4m3x4_to_bf16(w.x), a1 = e4m3x4_to_bf16(w.y), a2 = e4m3x4_to_bf16(w.z),
                        a3 = e4m3x4_to_bf16(w.w);
            if (y + kBatch < kMine) w = *reinterpret_cast<const uint4 *>(src + ((y + kBatch) * 128 + t) * 16);
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
        tiles += walk.count;
        if (C::kQBufs == 1 && ok && more) {   // once this segment's scores are done
          ok = split_q();
          more = ok && qwalk.next();
        }
      }
      if (!ok) give_up();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kFewIssuerWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool F8, int N, bool SEL>
cudaError_t launch_few_rows(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm,
                            int num_ctas, cudaStream_t stream) {
  using C = FewCfg<D, F8, N, SEL>;
  static std::mutex mu;
  static bool done[128] = {};
  const cudaError_t e = once_per_device(mu, done, [] {
    if (C::kShareRegs) {
      // the register shares come out of what the launch gets: a smaller launch would wait forever
      cudaFuncAttributes f;
      const cudaError_t got = cudaFuncGetAttributes(&f, few_rows_kernel<D, F8, N, SEL>);
      if (got != cudaSuccess) return got;
      if (f.numRegs != C::kRegsLaunch) return cudaErrorInvalidConfiguration;
    }
    return cudaFuncSetAttribute(few_rows_kernel<D, F8, N, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kDynamic);
  });
  if (e != cudaSuccess) return e;
  return launch_cooperative(few_rows_kernel<D, F8, N, SEL>, num_ctas, C::kThreads, C::kDynamic, stream, qm, km, vm, a);
}

}  // namespace
}  // namespace idx
