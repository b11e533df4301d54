// A token of every row of logits: temperature, top-k, top-p and min-p, drawn with given
// random numbers.
//
// Eight CTAs, a cluster, hold one row in shared memory: the logits are read once, and what
// the CTAs need of each other (maxima, histograms, sums, candidates) they read from each
// other's shared memory between cluster barriers.  Every CTA then finds the same thresholds
// from the same numbers; parameters come from the first CTA's copy, so that no barrier
// depends on memory that could change in between.
//
// A token may not depend on how sums are rounded, and a border (u Z between two tokens' sums,
// p Z between two masses) lies within 2^-24 of some sum in a percent of the rows.  So weights
// are integers, 2^44 exp((l - l_ref) / T) to about 2^-39 of itself or one unit; their sums are
// exact in 64 bits whatever the order, and the comparisons with p Z and u Z exact in 128.
//
// Thresholds: the kept tokens are a prefix of the order (logit descending, index ascending),
// so one number is enough, the composite (key, ~index) of the last kept one.  A first pass
// sorts the weights' exponents into bins of 1 / 32 octave, counts for top-k and leading bits
// of the weights for top-p; the elements of the bin that holds the border (for top-k those
// above as well) go into a list that every CTA gathers, and a radix descent over that list
// finds the composite.  Where the list is too long (many equal logits, a large k) the descent
// runs over the whole row, with the histograms of all CTAs.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <mutex>

#include "idx_device.cuh"
#include "kv_quant.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace idx {
namespace {

constexpr int kCtas = 8;         // of a cluster: a row
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRanges = kCtas * kWarps;   // a warp's part of the row
constexpr int kTile = 128;       // a warp's step: four elements a lane
constexpr uint32_t kKeyMasked = 0x007FFFFFu;   // radix_key(-inf)
constexpr int kOctaves = 44;     // below 2^-44 of the largest: no weight
constexpr int kCut = kOctaves * 256;
constexpr int kYBins = 1536;     // (D + 255) / 8 for D < kCut, three to a thread
constexpr int kDigit = 10;       // bits of a descent's level
constexpr int kBins = 1 << kDigit;
constexpr int kIndexBits = 19;
constexpr int kCompositeBits = 32 + kIndexBits;
static_assert(IDX_MAX_VOCAB <= 1 << kIndexBits, "an index in a composite");

// 2^(j / 256) in units of 2^-44: powers of 2^(1 / 256), multiplied up with 62 bits after the point.
struct Exp2Table {
  uint64_t v[256];
};
constexpr Exp2Table make_exp2_table() {
  Exp2Table t{};
  unsigned __int128 x = static_cast<unsigned __int128>(1) << 62;
  for (int j = 0; j < 256; ++j) {
    t.v[j] = static_cast<uint64_t>((x + (1ull << 17)) >> 18);
    x = (x * 0x402C6BE96AF2FB58ull + (1ull << 61)) >> 62;   // 2^(1 / 256)
  }
  return t;
}
__device__ const Exp2Table kExp2 = make_exp2_table();

constexpr float kMagic = 49152.0f;   // 1.5 * 2^15: a sum's last bit is 1 / 256

// How a row's logits become weights: exp(l / T) = 2^p with p = l c, c = log2(e) / T.
struct Row {
  float top;          // the largest logit
  float temperature;  // within 2^-60 .. 2^60
  float c_hi, c_lo;   // c in two terms
  float floor;        // of p: below it there is no weight
  int32_t top_bits;   // p + kMagic of the largest
  bool far;           // p would lose bits: differences to the largest are taken first
};

// p in two terms for two logits; the first is cut at r.floor (NaN and -inf as well).
__device__ __forceinline__ void exponents(float x0, float x1, const Row &r, uint64_t &p, uint64_t &lo) {
  float p0, p1;
  if (!r.far) {
    const uint64_t x = pack2(x0, x1), c = pack2(r.c_hi, r.c_hi);
    const uint64_t minus = mul2(x, pack2(-r.c_hi, -r.c_hi));
    lo = fma2(x, pack2(r.c_lo, r.c_lo), fma2(x, c, minus));
    p0 = fmaxf(-__uint_as_float(static_cast<uint32_t>(minus)), r.floor);
    p1 = fmaxf(-__uint_as_float(static_cast<uint32_t>(minus >> 32)), r.floor);
  } else {
    float l[2], q[2];
    const float v[2] = {x0, x1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // top - x = s + e exactly (Knuth's sum of two terms); an infinite top is no distance from itself
      const bool same = v[i] == r.top;
      const float s = same ? 0.0f : r.top - v[i], b = s - r.top, e = same ? 0.0f : (r.top - (s - b)) - (v[i] + b);
      const float m = s * r.c_hi;
      l[i] = -fmaf(e, r.c_hi, fmaf(s, r.c_lo, fmaf(s, r.c_hi, -m)));
      q[i] = fmaxf(-m, r.floor);
    }
    p0 = q[0];
    p1 = q[1];
    lo = pack2(l[0], l[1]);
  }
  p = pack2(p0, p1);
}
// p in steps of 1 / 256 below the largest's, >= 0.
__device__ __forceinline__ void steps(uint64_t p, const Row &r, uint64_t &t, int32_t (&d)[2]) {
  t = fma2(p, pack2(1.0f, 1.0f), pack2(kMagic, kMagic));
  d[0] = r.top_bits - static_cast<int32_t>(static_cast<uint32_t>(t));
  d[1] = r.top_bits - static_cast<int32_t>(static_cast<uint32_t>(t >> 32));
}

// Weights of two logits: 2^p is a power of two, a table entry of 8 bits and exp(g) - 1 of
// the rest g, |g| <= 2^-9.5, whose leading bits are kept apart so that integers hold it to
// 2^-40.  m: the weight before its shift by the power of two, 2^44 .. 2^45.  The last bit of
// a weight stands for all below it (it is always set), so roundings have no direction.
struct Weights {
  uint64_t w[2], m[2];
  int32_t d[2];
};
__device__ __forceinline__ void weights(float x0, float x1, const Row &r, const uint64_t *exp2_table, Weights &out) {
  constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
  constexpr float kHead = 0x1.8p-3f;    // 1.5 * 2^-3: a sum's last bit is 2^-26
  constexpr float kTail = 0x1.8p-17f;   // ... 2^-40
  uint64_t p, lo, t;
  exponents(x0, x1, r, p, lo);
  steps(p, r, t, out.d);
  const uint64_t one = pack2(1.0f, 1.0f), minus = pack2(-1.0f, -1.0f), ln2 = pack2(kLn2Hi, kLn2Hi);
  // p less its 256ths and its second term, again in two terms
  const uint64_t f0 = fma2(fma2(t, one, pack2(-kMagic, -kMagic)), minus, p), f = fma2(f0, one, lo);
  const uint64_t fl = fma2(fma2(f, minus, f0), one, lo);
  const uint64_t h = mul2(f, ln2);
  const uint64_t hl = fma2(fl, ln2, fma2(f, pack2(kLn2Lo, kLn2Lo), fma2(f, ln2, mul2(h, minus))));
  // exp(h + hl) - 1 = h + q
  const uint64_t q = fma2(mul2(h, h), fma2(h, pack2(1.0f / 6.0f, 1.0f / 6.0f), pack2(0.5f, 0.5f)), hl);
  const uint64_t head = fma2(h, one, pack2(kHead, kHead));
  const uint64_t rest = fma2(fma2(head, one, pack2(-kHead, -kHead)), minus, h);
  const uint64_t tail = fma2(fma2(q, one, rest), one, pack2(kTail, kTail));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t hb = static_cast<int32_t>(static_cast<uint32_t>(head >> (32 * i))) - __float_as_int(kHead);
    const int32_t tb = static_cast<int32_t>(static_cast<uint32_t>(tail >> (32 * i))) - __float_as_int(kTail);
    const int32_t g = (hb << 14) + tb;   // units of 2^-40
    const uint64_t b = exp2_table[-out.d[i] & 255];
    const uint64_t m = b + static_cast<uint64_t>((static_cast<int64_t>(static_cast<int32_t>(b >> 14)) * g) >> 26);
    out.m[i] = m;
    out.w[i] = out.d[i] < kCut ? m >> ((out.d[i] + 255) >> 8) | 1ull : 0ull;
  }
}
__device__ __forceinline__ uint64_t weight(float x, const Row &r, const uint64_t *exp2_table) {
  Weights v;
  weights(x, x, r, exp2_table, v);
  return v.w[0];
}

__device__ __forceinline__ uint32_t key_of(float x) { return x != x ? kKeyMasked : radix_key(x); }
__device__ __forceinline__ uint64_t composite(float x, int index) {
  return static_cast<uint64_t>(key_of(x)) << kIndexBits | static_cast<uint32_t>((1 << kIndexBits) - 1 - index);
}

template <typename T>
struct Quad;
template <>
struct Quad<float> {
  using Vec = float4;
  static constexpr int kListMost = 1024;   // a list that lies beside the row
  static __device__ __forceinline__ void get(const Vec &v, float (&x)[4]) {
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  }
  static __device__ __forceinline__ float one(float v) { return v; }
  static __device__ __forceinline__ float masked() { return -INFINITY; }
};
template <>
struct Quad<uint16_t> {
  using Vec = uint2;
  static constexpr int kListMost = 4096;   // bf16 rows are half as long, and their bins hold more equals
  static __device__ __forceinline__ void get(const Vec &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ float one(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ uint16_t masked() { return 0xFF80u; }
};

// What the CTAs of a row publish; every field is written before one barrier and read behind it.
template <typename T>
struct Shared {
  static constexpr int kSegment = Quad<T>::kListMost / 16;   // candidates of a warp
  // the first CTA's: the row's parameters
  float temperature, top_p, min_p, u;
  int32_t top_k, live;
  unsigned long long best;   // (key << 32) | ~index of the CTA's largest
  uint64_t all;              // its weights
  uint64_t above, kept;      // its weights above the border's bin, those that min-p keeps of them
  uint64_t sum;              // its kept weights, where no list gave them
  uint16_t count[kWarps];    // candidates
  uint16_t segment[kWarps][kSegment];   // their places in the warp's range, ascending
};

struct Found {
  uint32_t bin;
  uint64_t above, own;
};
// What a CTA uses alone.
struct Scratch {
  uint64_t warp_sum[kWarps];
  Found found;
  uint32_t overflow;
  uint64_t composite;
};

// The sum over the threads before this one, and over all.
__device__ __forceinline__ uint64_t exclusive_sum(uint64_t sum, Scratch &s, uint64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 31) s.warp_sum[warp] = upto;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s.warp_sum[w];
    total += s.warp_sum[w];
  }
  return before + upto - sum;
}

// A row's outputs.  log(w / Z) from the logit itself, whose weight may be a few units, and
// log1p of what the others weigh beside the largest.
__device__ void finish(const SampleArgs &a, int64_t row, int token, float x, uint64_t total, uint64_t top_weight, const Row &r) {
  a.token[row] = token;
  if (a.logprob == nullptr) return;
  const double y = x == r.top ? 0.0 : (static_cast<double>(r.top) - static_cast<double>(x)) / r.temperature;
  const double z = static_cast<double>(total - top_weight) / static_cast<double>(top_weight);
  a.logprob[row] = 0.0f - static_cast<float>(y) - log1pf(static_cast<float>(z));
}

// The element of this CTA's part of the row at which the kept weights pass `at`: the range,
// its step of a warp, the lane.  reach: the weights before the CTA's.  All its threads call.
template <typename T>
__device__ void pick(const SampleArgs &a, int64_t row, const T *data, int len, int rank, const uint64_t *warp_kept, uint64_t reach,
                     uint64_t at, uint64_t threshold, uint64_t least, uint64_t total, uint64_t top_weight, const Row &r,
                     const uint64_t *table, uint64_t *tile_sum) {
  using Q = Quad<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int range = 0;
  while (range < kWarps - 1 && at >= reach + warp_kept[range]) reach += warp_kept[range++];
  const int base = (rank * kWarps + range) * len;
  const auto tile = [&](int t, float (&x)[4], uint64_t (&w)[4]) {
    Q::get(*reinterpret_cast<const typename Q::Vec *>(data + range * len + t * kTile + 4 * lane), x);
    uint64_t sum = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Weights v;
      weights(x[2 * h], x[2 * h + 1], r, table, v);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 2 * h + i;
        w[k] = v.w[i] >= least && composite(x[k], base + t * kTile + 4 * lane + k) >= threshold ? v.w[i] : 0;
        sum += w[k];
      }
    }
    return sum;
  };
  const int tiles = len / kTile;
  for (int t = warp; t < tiles; t += kWarps) {
    float x[4];
    uint64_t w[4], sum = tile(t, x, w);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) tile_sum[t] = sum;
  }
  __syncthreads();
  int t = 0;
  while (t < tiles - 1 && at >= reach + tile_sum[t]) reach += tile_sum[t++];
  if (t % kWarps != warp) return;
  float x[4];
  uint64_t w[4];
  const uint64_t sum = tile(t, x, w);
  uint64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  uint64_t from = reach + upto - sum;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (at >= from && at < from + w[k]) finish(a, row, base + t * kTile + 4 * lane + k, x[k], total, top_weight, r);
    from += w[k];
  }
}

// The smallest integer that is not below p Z, 0 < p < 1: masses before kept tokens are below it.
__device__ __forceinline__ uint64_t ceil_product(float p, uint64_t z) {
  const uint64_t f = static_cast<uint64_t>(p * 0x1p64f);
  return __umul64hi(f, z) + (f == 0 || f * z != 0 ? 1 : 0);
}

__device__ __forceinline__ void clear_hist(uint32_t *hist) {
  for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) hist[i] = 0;
}
__device__ __forceinline__ void add_to_hist(uint32_t *hist, uint32_t bin, uint64_t w) {   // 64 bits from two words
  const uint32_t lo = static_cast<uint32_t>(w), was = atomicAdd(&hist[bin], lo);
  const uint32_t hi = static_cast<uint32_t>(w >> 32) + (was + lo < was ? 1u : 0u);
  if (hi != 0) atomicAdd(&hist[kBins + bin], hi);
}

// The bin of a descent's level, from the top, at which the running sum reaches want(total)
// (1 .. total).  One histogram, or those of all CTAs.  kMass: 64-bit sums in two words.
template <bool kMass, bool kAll, typename F>
__device__ __forceinline__ Found find_bin(uint32_t *hist, Scratch &s, F want) {
  constexpr int kPer = kBins / kThreads;
  static_assert(kPer == 2, "a thread's bins are one vector");
  const int first = kBins - kPer * (static_cast<int>(threadIdx.x) + 1);
  uint64_t own[kPer] = {}, total;
#pragma unroll
  for (int c = 0; c < (kAll ? kCtas : 1); ++c) {
    const uint32_t *const h = kAll ? cg::this_cluster().map_shared_rank(hist, c) : hist;
    const uint2 lo = *reinterpret_cast<const uint2 *>(h + first);
    own[0] += lo.x;
    own[1] += lo.y;
    if constexpr (kMass) {
      const uint2 hi = *reinterpret_cast<const uint2 *>(h + kBins + first);
      own[0] += static_cast<uint64_t>(hi.x) << 32;
      own[1] += static_cast<uint64_t>(hi.y) << 32;
    }
  }
  uint64_t above = exclusive_sum(own[0] + own[1], s, total);
  const uint64_t w = want(total);
#pragma unroll
  for (int i = kPer - 1; i >= 0; --i) {
    if (above < w && w <= above + own[i]) s.found = {static_cast<uint32_t>(first + i), above, own[i]};
    above += own[i];
  }
  __syncthreads();
  return s.found;
}

// The bin of exponents, from the largest, at which the running sum over all CTAs reaches
// want(total); bin kYBins where none does.  kMass: sums of weights' 16 leading bits.
template <bool kMass, typename F>
__device__ __forceinline__ Found find_exponent(uint32_t *hist, Scratch &s, F want) {
  constexpr int kPer = kYBins / kThreads;
  const int first = kPer * static_cast<int>(threadIdx.x);
  uint64_t own[kPer] = {}, sum = 0, total;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    const uint32_t *const h = cg::this_cluster().map_shared_rank(hist, c);
#pragma unroll
    for (int i = 0; i < kPer; ++i) own[i] += h[first + i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (kMass) own[i] = own[i] << 29 >> ((first + i) >> 5);
    sum += own[i];
  }
  if (threadIdx.x == 0) s.found = {kYBins, 0, 0};
  uint64_t above = exclusive_sum(sum, s, total);
  const uint64_t w = want(total);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (above < w && w <= above + own[i]) s.found = {static_cast<uint32_t>(first + i), above, own[i]};
    above += own[i];
  }
  __syncthreads();
  return s.found;
}

// The composite in list[0 .. n) at which the running sum, from the largest, over those >= low
// reaches want: of ones, or of weights.  The CTA alone.
template <bool kMass>
__device__ uint64_t descend_list(const uint64_t *list, int n, uint64_t low, uint64_t want, const Row &r,
                                 const uint64_t *table, uint32_t *hist, Scratch &s) {
  // the bits in which they differ
  if (threadIdx.x == 0) s.composite = 0;
  __syncthreads();
  const uint64_t any = list[0];
  uint64_t diff = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) diff |= list[i] ^ any;
  const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(diff >> 32));
  const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(diff));
  if ((threadIdx.x & 31) == 0 && (hi | lo) != 0) atomicOr(reinterpret_cast<unsigned long long *>(&s.composite), static_cast<unsigned long long>(hi) << 32 | lo);
  __syncthreads();
  int shift = 64 - __clzll(static_cast<long long>(s.composite));
  uint64_t prefix = any >> shift;
  while (shift > 0) {
    const int known = shift, bits = min(kDigit, shift);
    shift -= bits;
    clear_hist(hist);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t c = list[i];
      if (c < low || c >> known != prefix) continue;
      const uint32_t bin = static_cast<uint32_t>(c >> shift) & ((1u << bits) - 1);
      atomicAdd(&hist[2 * kBins + bin], 1u);
      if constexpr (kMass) add_to_hist(hist, bin, weight(radix_key_value(static_cast<uint32_t>(c >> kIndexBits)), r, table));
    }
    __syncthreads();
    const Found f = find_bin<kMass, false>(kMass ? hist : hist + 2 * kBins, s, [&](uint64_t) { return want; });
    prefix = prefix << bits | f.bin;
    want -= f.above;
    if (shift > 0 && hist[2 * kBins + f.bin] == 1) {   // one left: its other bits from the list
      for (int i = threadIdx.x; i < n; i += kThreads)
        if (list[i] >= low && list[i] >> shift == prefix) s.composite = list[i];
      __syncthreads();
      return s.composite;
    }
    __syncthreads();
  }
  return prefix;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  using Q = Quad<T>;
  using Vec = typename Q::Vec;
  using Pub = Shared<T>;
  constexpr int kListMost = Q::kListMost, kChunk = kListMost / kThreads;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint32_t *const hist = reinterpret_cast<uint32_t *>(smem_raw);                     // [3][kBins]
  uint64_t *const list = reinterpret_cast<uint64_t *>(hist + 3 * kBins);             // [kListMost] composites, by index
  T *const data = reinterpret_cast<T *>(list + kListMost);
  __shared__ Pub mine;
  __shared__ Scratch s;
  __shared__ uint64_t table[256];
  __shared__ unsigned long long warp_best[kWarps];
  __shared__ uint64_t warp_kept[kWarps], warp_above[kWarps];
  __shared__ uint64_t range_at[kRanges + 1], cta_above[kCtas], cta_kept[kCtas];
  __shared__ int32_t list_at[kRanges + 1];
  __shared__ uint64_t tile_sum[2 * kWarps];
  static_assert(kYBins <= 3 * kBins && kThreads * sizeof(uint64_t) <= 3 * kBins * sizeof(uint32_t), "what hist holds by turns");

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / kCtas;
  // this warp's range: [begin, begin + len) of the row, what lies past V masked
  const int len = a.warp_len;
  const int begin = (rank * kWarps + warp) * len;
  T *const own = data + warp * len;
  const T *const src = static_cast<const T *>(a.p.logits) + row * a.p.ld;

  for (int i = tid; i < 256; i += kThreads) table[i] = kExp2.v[i];
  clear_hist(hist);
  if (rank == 0 && tid == 0) {
    mine.live = a.p.rows == nullptr || row < *a.p.rows;
    mine.temperature = a.p.temperature != nullptr ? a.p.temperature[row] : 1.0f;
    mine.top_k = a.p.top_k != nullptr ? a.p.top_k[row] : 0;
    mine.top_p = a.p.top_p != nullptr ? a.p.top_p[row] : 1.0f;
    mine.min_p = a.p.min_p != nullptr ? a.p.min_p[row] : 0.0f;
    mine.u = a.p.u[row];
  }

  // the row, once, and its largest element (the first of several)
  float best_x = -INFINITY;
  int best_i = begin;
  constexpr int kFlight = 4;
  for (int t0 = 0; t0 < len; t0 += kFlight * kTile) {
    Vec v[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = begin + t0 + f * kTile + 4 * lane;
      T *const e = reinterpret_cast<T *>(&v[f]);
      if (a.vec && i + 4 <= a.p.V) {
        v[f] = __ldcs(reinterpret_cast<const Vec *>(src + i));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = i + k < a.p.V ? src[i + k] : Q::masked();
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int t = t0 + f * kTile + 4 * lane;
      if (t0 + f * kTile >= len) break;
      *reinterpret_cast<Vec *>(own + t) = v[f];
      float x[4];
      Q::get(v[f], x);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (x[k] > best_x) {
          best_x = x[k];
          best_i = begin + t + k;
        }
      }
    }
  }
  unsigned long long best = static_cast<unsigned long long>(key_of(best_x)) << 32 | static_cast<uint32_t>(~best_i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long b = __shfl_xor_sync(0xffffffffu, best, o);
    best = b > best ? b : best;
  }
  if (lane == 0) warp_best[warp] = best;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) best = warp_best[w] > best ? warp_best[w] : best;
    mine.best = best;
  }
  cluster.sync();
  best = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    const unsigned long long b = cluster.map_shared_rank(&mine, c)->best;
    best = b > best ? b : best;
  }
  const Pub *const params = cluster.map_shared_rank(&mine, 0);
  const float temperature = params->temperature, min_p = params->min_p, u = params->u;
  const float top_p = params->top_p < 1.0f ? params->top_p : 1.0f;   // NaN: off
  const int32_t top_k = params->top_k;
  const bool live = params->live != 0;
  const uint32_t top_key = static_cast<uint32_t>(best >> 32);

  // rows without a choice
  if (!live || top_key <= kKeyMasked || !(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f) {
    if (live && rank == 0 && tid == 0) {
      const bool empty = top_key <= kKeyMasked;
      a.token[row] = empty ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(best));
      if (a.logprob != nullptr) a.logprob[row] = empty ? -INFINITY : 0.0f;
    }
    cluster.sync();   // the others may still read this CTA's maximum
    return;
  }

  Row r;
  r.top = radix_key_value(top_key);
  r.temperature = fminf(fmaxf(temperature, 0x1p-60f), 0x1p60f);
  {
    const double c = 1.4426950408889634 / static_cast<double>(r.temperature);
    r.c_hi = static_cast<float>(c);
    r.c_lo = static_cast<float>(c - static_cast<double>(r.c_hi));
    // p keeps 2^-39 up to 2^10: the rounding of its second term is 2^-48 of it
    r.far = !(fabsf(r.top * r.c_hi) <= 1024.0f);
    r.floor = -INFINITY;
    uint64_t p, lo, t;
    int32_t d[2];
    exponents(r.top, r.top, r, p, lo);
    r.top_bits = 0;
    steps(p, r, t, d);
    r.top_bits = -d[0];
    r.floor = __uint_as_float(static_cast<uint32_t>(p)) - 64.0f;
  }
  const uint64_t top_weight = weight(r.top, r, table);
  uint64_t least = 1;   // of the weights that min-p keeps
  if (min_p > 0.0f) {
    const uint64_t f = static_cast<uint64_t>(fminf(min_p, 1.0f) * 0x1p63f);
    const uint64_t hi = __umul64hi(f, top_weight), lo = f * top_weight;
    least = (hi << 1 | lo >> 63) + (lo << 1 != 0 || f == 0 ? 1 : 0);
  }

  // f(tile, x[4]) over this warp's elements
  const auto each_tile = [&](auto f) {
    for (int t = 0; t < len; t += kTile) {
      float x[4];
      Q::get(*reinterpret_cast<const Vec *>(own + t + 4 * lane), x);
      f(t, x);
    }
  };

  uint64_t threshold = 0;   // composite of the last kept element
  uint64_t mass = 0;        // what top-p's border lies at
  bool count = top_k > 0 && top_k < a.p.V, whole = false;
  bool filter = count || top_p < 1.0f;
  Found y{kYBins, 0, 0};
  if (count) {
    each_tile([&](int, const float (&x)[4]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint64_t p, lo, t;
        int32_t d[2];
        exponents(x[2 * h], x[2 * h + 1], r, p, lo);
        steps(p, r, t, d);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (d[i] < kCut) atomicAdd(&hist[(d[i] + 255) >> 3], 1u);
      }
    });
    cluster.sync();
    y = find_exponent<false>(hist, s, [&](uint64_t total) {
      if (total <= static_cast<uint64_t>(top_k)) count = false;   // all that have a weight
      return static_cast<uint64_t>(top_k);
    });
    if (!count) {
      filter = top_p < 1.0f;
      cluster.sync();   // nobody reads the histogram any more
      clear_hist(hist);
      __syncthreads();
    }
  }
  if (filter && !count) {
    uint64_t sum = 0;
    each_tile([&](int, const float (&x)[4]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Weights v;
        weights(x[2 * h], x[2 * h + 1], r, table, v);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sum += v.w[i];
          if (v.d[i] < kCut) atomicAdd(&hist[(v.d[i] + 255) >> 3], static_cast<uint32_t>(v.m[i] >> 29) | 1u);
        }
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) warp_above[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) sum += warp_above[w];
      mine.all = sum;
    }
    cluster.sync();
    uint64_t z = 0;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) z += cluster.map_shared_rank(&mine, c)->all;
    mass = ceil_product(top_p, z);
    y = find_exponent<true>(hist, s, [&](uint64_t) { return mass; });
  }

  if (filter) {
    // candidates of the border in order of their index; the exact weights above its bin
    const int32_t bin = static_cast<int32_t>(y.bin);
    uint64_t above = 0, kept = 0;
    int32_t n = 0;
    each_tile([&](int t, const float (&x)[4]) {
      int32_t d[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint64_t p, lo, b;
        int32_t e[2];
        exponents(x[2 * h], x[2 * h + 1], r, p, lo);
        steps(p, r, b, e);
        d[2 * h] = (e[0] + 255) >> 3;
        d[2 * h + 1] = (e[1] + 255) >> 3;
      }
      uint32_t take = 0;
      bool over = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (d[k] == bin || (count && d[k] < bin)) take |= 1u << k;
        over = over || d[k] < bin;
      }
      if (!count && __any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          Weights v;
          weights(x[2 * h], x[2 * h + 1], r, table, v);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (d[2 * h + i] < bin) {
              above += v.w[i];
              kept += v.w[i] >= least ? v.w[i] : 0;
            }
          }
        }
      }
      if (__any_sync(0xffffffffu, take != 0)) {
        const int32_t here = __popc(take);
        int32_t upto = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int32_t up = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += up;
        }
        int32_t at = n + upto - here;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (take >> k & 1) {
            if (at < Pub::kSegment) mine.segment[warp][at] = static_cast<uint16_t>(t + 4 * lane + k);
            ++at;
          }
        }
        n += __shfl_sync(0xffffffffu, upto, 31);
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      above += __shfl_xor_sync(0xffffffffu, above, o);
      kept += __shfl_xor_sync(0xffffffffu, kept, o);
    }
    if (lane == 0) {
      warp_above[warp] = above;
      warp_kept[warp] = kept;
      mine.count[warp] = static_cast<uint16_t>(n);   // at most the warp's range
    }
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) {
        above += warp_above[w];
        kept += warp_kept[w];
      }
      mine.above = above;
      mine.kept = kept;
    }
    cluster.sync();

    // the list: places of the ranges, then the elements
    if (tid < kCtas) {
      cta_above[tid] = cluster.map_shared_rank(&mine, tid)->above;
      cta_kept[tid] = cluster.map_shared_rank(&mine, tid)->kept;
    }
    if (tid == 0) s.overflow = 0;
    __syncthreads();
    uint64_t listed;
    {
      const int32_t c = tid < kRanges ? cluster.map_shared_rank(&mine, tid / kWarps)->count[tid % kWarps] : 0;
      if (c > Pub::kSegment) s.overflow = 1;
      const uint64_t before = exclusive_sum(static_cast<uint64_t>(c), s, listed);
      if (tid <= kRanges) list_at[tid] = static_cast<int32_t>(before);
    }
    __syncthreads();
    n = static_cast<int32_t>(listed);
    whole = n == 0 || n > kListMost || s.overflow != 0;
    bool reading = false;   // the end of the barrier behind the last remote read is still to come
    if (!whole) {
      for (int i = tid; i < n; i += kThreads) {
        int w = 0;
#pragma unroll
        for (int step = kRanges / 2; step > 0; step >>= 1)
          if (list_at[w + step] <= i) w += step;
        const int c = w / kWarps, at = cluster.map_shared_rank(&mine, c)->segment[w % kWarps][i - list_at[w]];
        const float x = Q::one(cluster.map_shared_rank(data, c)[(w % kWarps) * len + at]);
        list[i] = composite(x, w * len + at);
      }
      cluster.barrier_arrive();
      reading = true;
      __syncthreads();
      const auto list_weight = [&](int i) { return weight(radix_key_value(static_cast<uint32_t>(list[i] >> kIndexBits)), r, table); };
      const auto list_mass = [&](uint64_t low) {
        uint64_t sum = 0, total;
        for (int i = tid; i < n; i += kThreads) sum += list[i] >= low ? list_weight(i) : 0;
        exclusive_sum(sum, s, total);
        __syncthreads();
        return total;
      };
      if (count) {
        if (rank != 0) {   // everything that is kept is in the first CTA's list as well
          cluster.barrier_wait();
          return;
        }
        threshold = descend_list<false>(list, n, 0, static_cast<uint64_t>(top_k), r, table, hist, s);
        if (top_p < 1.0f) {
          const uint64_t z = list_mass(threshold);
          threshold = descend_list<true>(list, n, threshold, ceil_product(top_p, z), r, table, hist, s);
        }
      } else {
        uint64_t over = 0;
#pragma unroll
        for (int c = 0; c < kCtas; ++c) over += cta_above[c];
        // the leading bits of the weights may have missed the bin
        if (over < mass && mass <= over + list_mass(0)) threshold = descend_list<true>(list, n, 0, mass - over, r, table, hist, s);
        else whole = true;
      }
      if (!whole) {
        // kept weights of the list: each thread's part of it, and up to each range
        uint64_t sum = 0, total, w[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          const int i = tid * kChunk + k;
          w[k] = 0;
          if (i < n && list[i] >= threshold) w[k] = list_weight(i);
          if (w[k] < least) w[k] = 0;
          sum += w[k];
        }
        uint64_t before = exclusive_sum(sum, s, total);
        const uint64_t f = u > 0.0f ? (u < 1.0f ? static_cast<uint64_t>(u * 0x1p64f) : ~0ull) : 0ull;
        if (count) {
          const uint64_t at = __umul64hi(f, total);
#pragma unroll
          for (int k = 0; k < kChunk; ++k) {
            if (at >= before && at < before + w[k]) {
              const uint64_t c = list[tid * kChunk + k];
              finish(a, row, (1 << kIndexBits) - 1 - static_cast<int>(c & ((1u << kIndexBits) - 1)),
                     radix_key_value(static_cast<uint32_t>(c >> kIndexBits)), total, top_weight, r);
            }
            before += w[k];
          }
          cluster.barrier_wait();
          return;
        }
        uint64_t *const part = reinterpret_cast<uint64_t *>(hist);   // the list's weights before each thread's
        part[tid] = before;
        __syncthreads();
        if (tid <= kRanges) {
          const int i = list_at[tid];
          uint64_t at = i / kChunk < kThreads ? part[i / kChunk] : total;
          for (int j = i / kChunk * kChunk; j < i && j < n; ++j) {
            if (list[j] < threshold) continue;
            const uint64_t v = list_weight(j);
            at += v >= least ? v : 0;
          }
          range_at[tid] = at;
        }
        __syncthreads();
        for (int c = 0; c < kCtas; ++c) total += cta_kept[c];
        const uint64_t at = __umul64hi(f, total);
        uint64_t reach = 0;
        for (int c = 0; c < rank; ++c) reach += cta_kept[c];
        reach += range_at[rank * kWarps];
        const uint64_t here = cta_kept[rank] + range_at[(rank + 1) * kWarps] - range_at[rank * kWarps];
        if (at >= reach && at < reach + here) {
          if (tid < kWarps) warp_kept[tid] += range_at[rank * kWarps + tid + 1] - range_at[rank * kWarps + tid];
          __syncthreads();
          pick<T>(a, row, data, len, rank, warp_kept, reach, at, threshold, least, total, top_weight, r, table, tile_sum);
        }
        cluster.barrier_wait();
        return;
      }
    }
    // long lists: the whole row, all CTAs
    if (reading) cluster.barrier_wait();
    uint64_t left = static_cast<uint64_t>(top_k), low = static_cast<uint64_t>(kKeyMasked + 1) << kIndexBits;
    for (int kind = count ? 0 : 1; kind < (top_p < 1.0f ? 2 : 1); ++kind) {   // top-k's border, top-p's
      uint64_t prefix = 0;
      for (int shift = kCompositeBits; shift > 0;) {
        const int known = shift, bits = min(kDigit, shift);
        shift -= bits;
        cluster.sync();   // nobody reads the histogram any more
        clear_hist(hist);
        __syncthreads();
        each_tile([&](int t, const float (&x)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t c = composite(x[k], begin + t + 4 * lane + k);
            if (c < low || c >> known != prefix) continue;
            const uint32_t at = static_cast<uint32_t>(c >> shift) & ((1u << bits) - 1);
            if (kind == 0) {
              atomicAdd(&hist[at], 1u);
            } else {
              const uint64_t w = weight(x[k], r, table);
              if (w != 0) add_to_hist(hist, at, w);
            }
          }
        });
        cluster.sync();
        const Found f = kind == 0 ? find_bin<false, true>(hist, s, [&](uint64_t) { return left; })
                                  : find_bin<true, true>(hist, s, [&](uint64_t z) {
                                      if (known == kCompositeBits) left = ceil_product(top_p, z);
                                      return left;
                                    });
        prefix = prefix << bits | f.bin;
        left -= f.above;
      }
      threshold = low = prefix;
    }
    cluster.sync();
  }

  // the kept weights of the row
  uint64_t sum = 0;
  each_tile([&](int t, const float (&x)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Weights v;
      weights(x[2 * h], x[2 * h + 1], r, table, v);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (v.w[i] >= least && (threshold == 0 || composite(x[2 * h + i], begin + t + 4 * lane + 2 * h + i) >= threshold)) sum += v.w[i];
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) warp_kept[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) sum += warp_kept[w];
    mine.sum = sum;
  }
  cluster.sync();
  uint64_t total = 0, reach = 0, here = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    const uint64_t v = cluster.map_shared_rank(&mine, c)->sum;
    if (c < rank) reach += v;
    if (c == rank) here = v;
    total += v;
  }
  cluster.barrier_arrive();
  const uint64_t at = __umul64hi(u > 0.0f ? (u < 1.0f ? static_cast<uint64_t>(u * 0x1p64f) : ~0ull) : 0ull, total);
  if (at >= reach && at < reach + here)
    pick<T>(a, row, data, len, rank, warp_kept, reach, at, threshold, least, total, top_weight, r, table, tile_sum);
  cluster.barrier_wait();
}

template <typename T>
constexpr size_t fixed_smem() {
  return 3 * kBins * sizeof(uint32_t) + Quad<T>::kListMost * sizeof(uint64_t);
}

template <typename T>
cudaError_t launch(SampleArgs a, cudaStream_t stream) {
  constexpr int kSpan = kCtas * kWarps * kTile;
  constexpr int kMost = static_cast<int>(fixed_smem<T>()) + IDX_MAX_VOCAB / kCtas * static_cast<int>(sizeof(T));
  static_assert(IDX_MAX_VOCAB % kSpan == 0 && IDX_MAX_VOCAB / kRanges / kTile <= 2 * kWarps, "whole steps of every warp");
  static std::mutex mu;
  static bool done[128];
  cudaError_t e = once_per_device(mu, done, [] {
    return cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  });
  if (e != cudaSuccess) return e;
  a.warp_len = static_cast<int32_t>((a.p.V + kSpan - 1) / kSpan) * kTile;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {kCtas, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.p.R) * kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = fixed_smem<T>() + static_cast<size_t>(kWarps) * a.warp_len * sizeof(T);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
  return a.p.logits_dtype == IDX_LOGITS_F32 ? launch<float>(a, stream) : launch<uint16_t>(a, stream);
}

}  // namespace idx
