// A token of every row of logits: temperature, top-k, top-p and min-p, drawn with given
// random numbers.
//
// A cluster of up to eight CTAs holds one row in shared memory: the logits are read once.  What
// the CTAs need of each other (maxima, sums, histograms by octave, counts) each writes into
// all of them before a cluster barrier, so that behind it nobody waits for another SM; only
// one octave's bins and the candidates are read from afar.  Every CTA then finds the same
// border from the same numbers; parameters come from the first CTA's copy, so that no
// barrier depends on memory that could change in between.
//
// A token may not depend on how sums are rounded, and a border (u Z between two tokens' sums,
// p Z between two masses) lies within 2^-24 of some sum in a percent of the rows.  So weights
// are integers, 2^44 exp(l / T) over the power of two at or above the largest exp(l / T), to
// about 2^-38 of itself or one unit; their sums are exact in 64 bits whatever the order, and
// the comparisons with p Z and u Z exact in 128.
//
// Thresholds: the kept tokens are a prefix of the order (logit descending, index ascending),
// so one number is enough, the composite (key, ~index) of the last kept one.  A first pass
// sorts the weights' exponents into bins of 1 / 64 octave, counts for top-k and leading bits
// of the weights for top-p; the elements of the bin that holds the border (for top-k those
// above as well, where they are few) go into a list that the first CTA gathers and searches, and
// what lies above it is summed exactly.  (Leading bits can point at the neighbour of a bin whose edge
// is next to the border; the exact sum tells, and the neighbour is taken.)  A bin with too many is cut into 128 finer ones first; where even those hold too many (equal
// logits), a radix descent runs over the whole row.  (Descents over the whole row for every
// border took 953 us for 256 rows of 151,552 fp32 logits of mixed width, most with top-p; this 194 to 212,
// by the parameters that the rows draw.)
//
// What bounds it: reading those rows would take 22.9 us at the measured copy bandwidth.  Their
// weights to 2^-38 are some 30 instructions a logit, 27 us if every slot were used.  The rest is the
// chain of a row's steps, 25 to 30 us with two rows to an SM, in which warps wait for the slowest
// one of the cluster (issue slots 44% busy, a third of the stalls at barriers).  A single row with
// top-p of 151,552 logits takes some 40,000 cycles: reading and the largest logit 6,400, weights
// and histogram 12,000, border, candidates and what lies above 10,800, the list 6,200 and the token
// among the kept ones 4,400.  22,800 of them are passes over the 37 logits of a thread, not latency.
// Without filters it takes 20,000: reading 6,000, weights 7,600, their sums over the cluster 1,200, the
// token 5,100.  (Sums above from a histogram of two words to a bin of 1 / 32 octave, off by 2^-33, took
// 203 to 225 us on the 256 rows' inputs, and a row's last bits depended on its CTAs; exact ones beside
// that histogram 216 to 243.)
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "idx_device.cuh"
#include "kv_quant.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace idx {
namespace {

constexpr int kCtas = 8;         // of a cluster, a row, at most
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRanges = kCtas * kWarps;   // warps' parts of the row
constexpr int kTile = 128;       // a warp's step: four elements a lane
constexpr uint32_t kKeyMasked = 0x007FFFFFu;   // radix_key(-inf)
constexpr int kFine = 128;       // parts of a bin of exponents
constexpr int kOctaves = 44;     // below 2^-44 of the largest's octave: no weight
constexpr int kCut = kOctaves * 64;
constexpr int kOctaveBins = 48;  // octaves, with room
constexpr int kYBins = kOctaveBins * 64;   // d + 63 for d < kCut, 64 to an octave
constexpr int kDigit = 9;        // bits of a descent's level
constexpr int kBins = 1 << kDigit;
constexpr int kSmallList = 256;  // searched by two or four threads per element
constexpr int kIndexBits = 19;
constexpr int kCompositeBits = 32 + kIndexBits;
static_assert(IDX_MAX_VOCAB <= 1 << kIndexBits, "an index in a composite");

// 2^(j / 64) = t 2^-25 2^-off: 26 bits that a product with them loses nothing of, and what
// they miss by.  Powers of 2^(1 / 64), multiplied up with 62 bits after the point.
struct Exp2 {
  int32_t t;
  float off;
};
struct Exp2Table {
  Exp2 v[64];
};
constexpr Exp2Table make_exp2_table() {
  Exp2Table table{};
  unsigned __int128 x = static_cast<unsigned __int128>(1) << 62;
  for (int j = 0; j < 64; ++j) {
    const uint64_t v = static_cast<uint64_t>(x), t = (v + (1ull << 36)) >> 37;
    const double miss = static_cast<double>(static_cast<int64_t>((t << 37) - v)) / static_cast<double>(v);
    table.v[j] = {static_cast<int32_t>(t), static_cast<float>(miss * 1.4426950408889634)};
    x = (x * 0x40B268F9DE0183BAull + (1ull << 61)) >> 62;   // 2^(1 / 64)
  }
  return table;
}
__device__ const Exp2Table kExp2 = make_exp2_table();
constexpr int kColumns = 16;   // the table stands in 16 columns of two banks: a lane reads its own

constexpr float kMagic = 196608.0f;   // 1.5 * 2^17: a sum's last bit is 1 / 64

// How a row's logits become weights: exp(l / T) = 2^p up to a factor of the row, with
// p = (l - ref) c, c = log2(e) / T.  ref is 0 while p stays small enough for the second term
// that its product has, else the largest logit: then every logit with a weight lies within
// a factor of two of it, and the difference is exact.
struct Row {
  float top;            // the largest logit
  float ref;
  float temperature;    // within 2^-60 .. 2^60
  float c_hi, c_lo;     // c in two terms
  uint32_t whole_bits;  // p + kMagic of the largest, up to a whole octave: weights are relative to that
  uint64_t least;       // of the weights that min-p keeps
};

// -p for two logits, in two terms (p = -(minus) + lo).
__device__ __forceinline__ void exponents(float x0, float x1, const Row &r, uint64_t &minus, uint64_t &lo) {
  const uint64_t x = fma2(pack2(x0, x1), pack2(1.0f, 1.0f), pack2(-r.ref, -r.ref));
  minus = mul2(x, pack2(-r.c_hi, -r.c_hi));
  lo = fma2(x, pack2(r.c_lo, r.c_lo), fma2(x, pack2(r.c_hi, r.c_hi), minus));
}
// p to 64ths, as the bits of a float: they ascend with p, from kMagic's for 0 by one a 64th.
__device__ __forceinline__ uint64_t to_64ths(uint64_t minus) { return fma2(minus, pack2(-1.0f, -1.0f), pack2(kMagic, kMagic)); }
// 64ths below the largest's octave for each.  Unsigned: negative floats and NaN end up far behind
// kCut as well.
__device__ __forceinline__ void steps(uint64_t t, const Row &r, uint32_t (&d)[2]) {
  d[0] = r.whole_bits - static_cast<uint32_t>(t);
  d[1] = r.whole_bits - static_cast<uint32_t>(t >> 32);
}

// A bin of exponents for d 64ths, kFar for what has no weight.
constexpr int32_t kFar = 1 << 20;
__device__ __forceinline__ int32_t exponent_bin(uint32_t d) { return d < kCut ? static_cast<int32_t>(d + 63) : kFar; }
// The part of its bin that element i of a pair lies in, behind the bin: smaller above.
__device__ __forceinline__ int32_t fine_code(uint64_t minus, uint64_t t, uint32_t d, int i) {
  if (d >= kCut) return kFar * kFine;
  const float v = __uint_as_float(static_cast<uint32_t>(minus >> (32 * i))), c = __uint_as_float(static_cast<uint32_t>(t >> (32 * i)));
  const float f = (kMagic - c) - v;   // exact, within 2^-7: 128 parts of a 64th
  const int32_t part = min(max(static_cast<int32_t>((f + 0x1p-7f) * 0x1p13f), 0), kFine - 1);
  return static_cast<int32_t>(d + 63) * kFine + (kFine - 1 - part);
}

// Weights of two logits: 2^p is a power of two, a table entry of 6 bits and exp(g) - 1 of
// the rest g, |g| <= 2^-7.5, whose leading term is kept apart so that integers hold it to
// 2^-37.  m: the weight before its shift by the power of two, 2^62 .. 2^63.  The last bit
// of a weight stands for all below it (it is always set), so roundings have no direction.
// Measured against 64 bits: off by 2^-38.2 in the mean square, 2^-36.2 at most.
struct Weights {
  uint64_t w[2], m[2];   // w: of no meaning from kCut on
  uint32_t d[2];
};
__device__ __forceinline__ void weights(float x0, float x1, const Row &r, const Exp2 *table, Weights &out) {
  constexpr float kLn2 = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
  constexpr float kTail = 0x1.8p-14f;     // 1.5 * 2^-14: a sum's last bit is 2^-37
  uint64_t minus, lo;
  exponents(x0, x1, r, minus, lo);
  const uint64_t t = to_64ths(minus), one = pack2(1.0f, 1.0f), negative = pack2(-1.0f, -1.0f), ln2 = pack2(kLn2, kLn2);
  steps(t, r, out.d);
  // (kMagic's last six bits are 0, and so are the octave's)
  const uint32_t column = threadIdx.x & (kColumns - 1);
  const Exp2 e0 = table[(static_cast<uint32_t>(t) & 63u) * kColumns | column], e1 = table[(static_cast<uint32_t>(t >> 32) & 63u) * kColumns | column];
  lo = pack2(__uint_as_float(static_cast<uint32_t>(lo)) - e0.off, __uint_as_float(static_cast<uint32_t>(lo >> 32)) - e1.off);
  const uint64_t f = fma2(minus, negative, fma2(t, negative, pack2(kMagic, kMagic)));   // p less its 64ths
  // exp((f + lo) ln 2) - 1 = h + q, with h + b = (f + lo) ln 2
  const uint64_t mh = mul2(f, pack2(-kLn2, -kLn2));   // -h
  const uint64_t b = fma2(lo, ln2, fma2(f, pack2(kLn2Lo, kLn2Lo), fma2(f, ln2, mh)));
  const uint64_t g = fma2(mh, negative, b);
  const uint64_t a = fma2(g, fma2(g, pack2(1.0f / 24.0f, 1.0f / 24.0f), pack2(1.0f / 6.0f, 1.0f / 6.0f)), pack2(0.5f, 0.5f));
  const uint64_t tail = fma2(fma2(mul2(g, g), a, b), one, pack2(kTail, kTail));
  const uint64_t head = mul2(mh, pack2(-0x1p37f, -0x1p37f));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t gi = __float2int_rn(__uint_as_float(static_cast<uint32_t>(head >> (32 * i)))) +
                       (static_cast<int32_t>(static_cast<uint32_t>(tail >> (32 * i))) - __float_as_int(kTail));
    const int32_t e = i == 0 ? e0.t : e1.t;
    const uint64_t w = (static_cast<uint64_t>(static_cast<uint32_t>(e) << 5) << 32) + static_cast<uint64_t>(static_cast<int64_t>(e) * gi);
    out.m[i] = w;
    out.w[i] = w >> ((out.d[i] + 63 + 18 * 64) >> 6) | 1ull;
  }
}
__device__ __noinline__ uint64_t weight(float x, const Row &r, const Exp2 *table) {   // one, where they are few
  Weights v;
  weights(x, x, r, table, v);
  return v.d[0] < kCut ? v.w[0] : 0;
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
  static __device__ __forceinline__ float one(float v) { return v; }
  static constexpr int kListMost = 768;    // candidates of a row in the list
  static __device__ __forceinline__ void get(const Vec &v, float (&x)[4]) {
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  }
  static __device__ __forceinline__ float masked() { return -INFINITY; }
};
template <>
struct Quad<uint16_t> {
  using Vec = uint2;
  static __device__ __forceinline__ float one(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static constexpr int kListMost = 4096;   // bf16 rows are half as long, and their bins hold more equals
  static __device__ __forceinline__ void get(const Vec &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint16_t masked() { return 0xFF80u; }
};

// What the CTAs of a row tell each other: each writes its own entry into every CTA, before a
// barrier that all read behind, so that nobody waits for another SM's shared memory.
struct Told {
  unsigned long long best;   // (key << 32) | ~index of the CTA's largest
  uint64_t all;              // its weights
  uint64_t above, kept;      // its weights (or elements) above the border's bin, the weights that min-p keeps of them
  uint64_t sum;              // its kept weights, where no list gave them
};
struct Params {              // of the row, from the first CTA
  float temperature, c_hi, c_lo, top_p, min_p, u;
  int32_t top_k, live;
};
struct Verdict {             // on a list, from the first CTA
  uint64_t threshold;        // composite of the last kept element
  uint64_t total, at;        // kept weights of the row; of the CTA `owner`, what the drawn token's pass
  int32_t owner;             // -1: the border was not in the list
};
template <typename T, bool kList>
struct Shared {
  static constexpr int kSegment = kList ? Quad<T>::kListMost / 16 : 1;   // candidates of a warp
  Told told[kCtas];
  Params params;
  Verdict verdict;
  float octave[kCtas][kOctaveBins];      // sums of the exponents' bins
  uint16_t count[kRanges];               // candidates of every warp
  T logit[kWarps][kSegment];             // this CTA's, and their places in the warp's range, by place
  uint16_t place[kWarps][kSegment];
};

struct Found {
  uint32_t bin;
  uint64_t above, own;
};
// What a CTA uses alone.
struct Scratch {
  uint64_t warp_sum[kWarps];
  alignas(8) float bin[64];
  Found found;
  uint64_t composite;
};

// The sum over the threads before this one, and over all.
struct Sums {
  uint64_t before, all;
};
__device__ __noinline__ Sums exclusive_sum(uint64_t v, uint64_t *warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  // every warp sums the warps' sums, one a lane
  uint64_t w = lane < kWarps ? warp_sum[lane] : 0;
  const uint64_t own = w;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += up;
  }
  Sums r;
  r.before = __shfl_sync(0xffffffffu, w - own, warp) + upto - v;
  r.all = __shfl_sync(0xffffffffu, w, kWarps - 1);
  return r;
}

__device__ __forceinline__ uint64_t warp_total(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The sum of a value per warp, for one warp to call.
__device__ __forceinline__ uint64_t warps_total(const uint64_t *v) {
  return warp_total((threadIdx.x & 31) < kWarps ? v[threadIdx.x & 31] : 0);
}

// A row's outputs.  log(w / Z) from the logit itself, whose weight may be a few units, and
// log1p of what the others weigh beside the largest.
__device__ __noinline__ void finish(const SampleArgs &a, int64_t row, int token, float x, uint64_t total, const Row &r, const Exp2 *table) {
  a.token[row] = token;
  if (a.logprob == nullptr) return;
  const float y = x == r.top ? 0.0f : (r.top - x) / r.temperature;
  const uint64_t top = weight(r.top, r, table);
  const float z = static_cast<float>(total - top) / static_cast<float>(top);
  a.logprob[row] = 0.0f - y - log1pf(z);
}

// The element of this CTA's part of the row at which the kept weights pass `at`: the range,
// its step of a warp, the lane.  reach: the weights before the CTA's.  All its threads call.
template <typename T>
__device__ __noinline__ void pick(const SampleArgs &a, int64_t row, const T *data, int rank, const uint64_t *warp_kept, uint64_t reach,
                                  uint64_t at, uint64_t threshold, uint64_t total, const Row &r, const Exp2 *table, uint64_t *tile_sum) {
  using Q = Quad<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, len = a.warp_len, tiles = len / kTile;
  // the last entry v[i], i < n <= 32, before which there is no more than `at` (and what is before it): for every warp by itself
  const auto reached = [&](const uint64_t *v, int n) {
    const uint64_t own = lane < n ? v[lane] : 0;
    uint64_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, at < reach + upto);
    const int i = min(past != 0 ? __ffs(past) - 1 : 31, n - 1);
    reach += __shfl_sync(0xffffffffu, upto - own, i);
    return i;
  };
  const int range = reached(warp_kept, kWarps), base = (rank * kWarps + range) * len;
  float x[4];
  uint64_t w[4], sum = 0;
  const auto step = [&](int t) {
    Q::get(*reinterpret_cast<const typename Q::Vec *>(data + range * len + t * kTile + 4 * lane), x);
    sum = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Weights v;
      weights(x[2 * h], x[2 * h + 1], r, table, v);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 2 * h + i;
        w[k] = v.d[i] < kCut && v.w[i] >= r.least && composite(x[k], base + t * kTile + 4 * lane + k) >= threshold ? v.w[i] : 0;
        sum += w[k];
      }
    }
  };
  // the sums of all steps, a warp a step, then within the one that has it
  int t = warp;
#pragma unroll 1
  for (int n = warp; n < tiles; n += kWarps) {
    t = n;
    step(t);
    const uint64_t all = warp_total(sum);
    if (lane == 0) tile_sum[t] = all;
  }
  __syncthreads();
  const int chosen = reached(tile_sum, tiles);
  if (chosen % kWarps != warp) return;
  if (chosen != t) step(chosen);   // the last step's are still there
  uint64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  uint64_t from = reach + upto - sum;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (at >= from && at < from + w[k]) {
      finish(a, row, base + chosen * kTile + 4 * lane + k, x[k], total, r, table);
      return;
    }
    from += w[k];
  }
}

// The smallest integer that is not below p Z, 0 < p < 1: masses before kept tokens are below it.
__device__ __forceinline__ uint64_t ceil_product(float p, uint64_t z) {
  const uint64_t f = static_cast<uint64_t>(p * 0x1p64f);
  return __umul64hi(f, z) + (f == 0 || f * z != 0 ? 1 : 0);
}

__device__ __forceinline__ void clear_hist(uint32_t *hist, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) hist[i] = 0;
}
__device__ __forceinline__ void add_to_hist(uint32_t *hist, uint32_t bin, uint64_t w) {   // 64 bits from two words
  const uint32_t lo = static_cast<uint32_t>(w), was = atomicAdd(&hist[bin], lo);
  const uint32_t hi = static_cast<uint32_t>(w >> 32) + (was + lo < was ? 1u : 0u);
  if (hi != 0) atomicAdd(&hist[kBins + bin], hi);
}

// The bin of a descent's level, from the top, at which the running sum reaches `want`
// (1 .. the sum of all; bin kBins where none does).  One histogram, or those of all CTAs;
// mass: 64-bit sums in two words.
__device__ __noinline__ Found find_bin(bool mass, int ctas, uint32_t *hist, Scratch &s, uint64_t want) {
  static_assert(kBins == kThreads, "a bin a thread");
  const int bin = kBins - 1 - static_cast<int>(threadIdx.x);
  uint64_t own = 0;
  if (threadIdx.x == 0) s.found = {kBins, 0, 0};
#pragma unroll 1
  for (int c = 0; c < ctas; ++c) {
    const uint32_t *const h = ctas > 1 ? cg::this_cluster().map_shared_rank(hist, c) : hist;
    own += h[bin];
    if (mass) own += static_cast<uint64_t>(h[kBins + bin]) << 32;
  }
  const uint64_t above = exclusive_sum(own, s.warp_sum).before;
  if (above < want && want <= above + own) s.found = {static_cast<uint32_t>(bin), above, own};
  __syncthreads();
  return s.found;
}

// The octaves' sums of this CTA's bins of exponents, to all CTAs: octave[rank] there.
__device__ __noinline__ void push_octaves(const uint32_t *hist, float (*octave)[kOctaveBins]) {
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = warp; o < kOctaveBins; o += kWarps) {
    const float v = static_cast<float>(__reduce_add_sync(0xffffffffu, hist[o * 64 + lane] + hist[o * 64 + 32 + lane]));
    const cg::cluster_group cluster = cg::this_cluster();
    if (lane < cluster.num_blocks()) cluster.map_shared_rank(octave, lane)[cluster.block_rank()][o] = v;
  }
}

// Of 32 values, one a lane, the first at which the running sum reaches `want` (the last that
// is not 0 if none does), and the sum before it; `all`: of all.
struct Reached {
  int at;
  float before, all;
};
__device__ __forceinline__ Reached reach_in_warp(float v, float want) {
  const int lane = threadIdx.x & 31;
  float upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  const uint32_t there = __ballot_sync(0xffffffffu, upto >= want && v != 0.0f), some = __ballot_sync(0xffffffffu, v != 0.0f);
  Reached r;
  r.at = there != 0 ? __ffs(there) - 1 : some != 0 ? 31 - __clz(some) : 31;
  r.before = __shfl_sync(0xffffffffu, upto - v, r.at);
  r.all = __shfl_sync(0xffffffffu, upto, 31);
  return r;
}

// The bin of exponents, from the largest, at which the running sum over all CTAs reaches
// `want`, and the sum of all: first the octave, then its bin, so that a thread reads one bin
// of another CTA.  In fp32: counts below 2^24 are exact; masses may miss a border next to an end
// of its bin, which the exact sums behind it find out.
struct Exponent {
  int32_t bin;
  float all;
};
__device__ __noinline__ Exponent find_exponent(bool mass, const uint32_t *hist, const float (*octave)[kOctaveBins], float *sum,
                                               float want) {
  static_assert(kOctaveBins > 32 && kOctaveBins <= 64, "one or two octaves a lane");
  const int tid = threadIdx.x, lane = tid & 31, ctas = static_cast<int>(cg::this_cluster().num_blocks());
  const auto scaled = [&](float v, int o) { return mass ? v * __uint_as_float(static_cast<uint32_t>(127 - o) << 23) : v; };
  float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    v0 += octave[c][lane];
    if (lane + 32 < kOctaveBins) v1 += octave[c][lane + 32];
  }
  Reached r = reach_in_warp(scaled(v0, lane), want);
  const Reached far = reach_in_warp(scaled(v1, lane + 32), want - r.all);
  Exponent e;
  e.all = r.all + far.all;
  int o = r.at;
  float before = r.before;
  if (r.all < want && far.all != 0.0f) {
    o = 32 + far.at;
    before = r.all + far.before;
  }
  static_assert(64 * kCtas == kThreads, "a bin of a CTA a thread");
  const int c = tid & (kCtas - 1), b = tid / kCtas;
  float v = c < ctas ? static_cast<float>(cg::this_cluster().map_shared_rank(hist, c)[o * 64 + b]) : 0.0f;
#pragma unroll
  for (int k = kCtas / 2; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  if (c == 0) sum[b] = scaled(v, o);
  __syncthreads();
  const float2 two = reinterpret_cast<const float2 *>(sum)[lane];   // two neighbours a lane
  const Reached pair = reach_in_warp(two.x + two.y, want - before);
  const float x = __shfl_sync(0xffffffffu, two.x, pair.at), y = __shfl_sync(0xffffffffu, two.y, pair.at);
  e.bin = o * 64 + 2 * pair.at + (pair.before + x < want - before && y != 0.0f ? 1 : 0);
  return e;
}

// The composite in list[0 .. n) at which the running sum, from the largest, over those >= low
// reaches want: of ones, or of weights.  The CTA alone.
__device__ __noinline__ uint64_t descend_list(bool mass, const uint64_t *list, int n, uint64_t low, uint64_t want, const Row &r,
                                 const Exp2 *table, uint32_t *hist, Scratch &s) {
  // the bits in which they differ
  if (threadIdx.x == 0) s.composite = 0;
  __syncthreads();
  const uint64_t any = list[0];
  uint64_t diff = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) diff |= list[i] ^ any;
  const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(diff >> 32));
  const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(diff));
  if ((threadIdx.x & 31) == 0 && (hi | lo) != 0)
    atomicOr(reinterpret_cast<unsigned long long *>(&s.composite), static_cast<unsigned long long>(hi) << 32 | lo);
  __syncthreads();
  int shift = 64 - __clzll(static_cast<long long>(s.composite));
  uint64_t prefix = any >> shift;
  while (shift > 0) {
    const int known = shift, bits = min(kDigit, shift);
    shift -= bits;
    clear_hist(hist, 3 * kBins);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t c = list[i];
      if (c < low || c >> known != prefix) continue;
      const uint32_t bin = static_cast<uint32_t>(c >> shift) & ((1u << bits) - 1);
      atomicAdd(&hist[2 * kBins + bin], 1u);
      if (mass) add_to_hist(hist, bin, weight(radix_key_value(static_cast<uint32_t>(c >> kIndexBits)), r, table));
    }
    __syncthreads();
    const Found f = find_bin(mass, 1, mass ? hist : hist + 2 * kBins, s, want);
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

// The histogram, in its second half the list, the row; without filters the row alone.
constexpr size_t kListOffset = 3 * kBins * sizeof(uint32_t);
template <typename T, bool kList>
__host__ __device__ constexpr size_t fixed_smem() {
  constexpr size_t list = kListOffset + Quad<T>::kListMost * sizeof(uint64_t), hist = kYBins * sizeof(uint32_t);
  return !kList ? 0 : list > hist ? list : hist;
}

// kTopK, kTopP: the rows may have these filters.
template <typename T, bool kTopK, bool kTopP>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  using Q = Quad<T>;
  using Vec = typename Q::Vec;
  using Pub = Shared<T, kTopK || kTopP>;
  constexpr int kListMost = Q::kListMost, kChunk = (kListMost + kThreads - 1) / kThreads;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint32_t *const hist = reinterpret_cast<uint32_t *>(smem_raw);                     // [kYBins], [3][kBins] in descents
  uint64_t *const list = reinterpret_cast<uint64_t *>(smem_raw + kListOffset);  // [kListMost] composites, by index
  T *const data = reinterpret_cast<T *>(smem_raw + fixed_smem<T, kTopK || kTopP>());
  __shared__ Pub mine;
  __shared__ Scratch s;
  __shared__ Row r;
  __shared__ __align__(8) Exp2 table[64 * kColumns];
  __shared__ unsigned long long warp_best[kWarps];
  __shared__ uint64_t warp_kept[kWarps], warp_above[kWarps];
  __shared__ uint64_t cta_at[kCtas + 1];
  __shared__ int32_t list_at[kRanges + 1];
  __shared__ uint64_t tile_sum[2 * kWarps];
  static_assert(kYBins >= 3 * kBins && kThreads * sizeof(uint64_t) <= kListOffset && kFine <= kBins, "what hist holds by turns");

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = a.ctas;   // a power of two
  const int64_t row = blockIdx.x >> (__ffs(ctas) - 1);
  // this warp's range: [begin, begin + len) of the row, what lies past V masked
  const int len = a.warp_len;
  const int begin = (rank * kWarps + warp) * len;
  T *const own = data + warp * len;
  const T *const src = static_cast<const T *>(a.p.logits) + row * a.p.ld;

  cluster.barrier_arrive();
  grid_dependency_trigger();
  for (int i = tid; i < 64 * kColumns; i += kThreads) table[i] = kExp2.v[i / kColumns];
  // what CTAs that are not there would tell
  if (tid >= ctas && tid < kCtas) mine.told[tid] = Told{};
  if constexpr (kTopK || kTopP) {
    for (int i = ctas * kOctaveBins + tid; i < kCtas * kOctaveBins; i += kThreads) (&mine.octave[0][0])[i] = 0.0f;
    if (tid >= ctas * kWarps && tid < kRanges) mine.count[tid] = 0;
    clear_hist(hist, kYBins);
  }
  grid_dependency_wait();
  Params par{};
  if (rank == 0 && warp == 0) {   // every lane the same; used behind the row's loads
    par.live = a.p.rows == nullptr || row < *a.p.rows;
    par.temperature = a.p.temperature != nullptr ? a.p.temperature[row] : 1.0f;
    par.top_k = kTopK ? a.p.top_k[row] : 0;
    par.top_p = kTopP ? a.p.top_p[row] : 1.0f;
    par.min_p = a.p.min_p != nullptr ? a.p.min_p[row] : 0.0f;
    par.u = a.p.u[row];
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
  if (rank == 0 && warp == 0) {
    // c = log2(e) / T in two terms
    constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f;
    const float T_used = fminf(fmaxf(par.temperature, 0x1p-60f), 0x1p60f);
    par.c_hi = kHi / T_used;
    par.c_lo = (fmaf(-par.c_hi, T_used, kHi) + kLo) / T_used;
  }
  __syncthreads();
  if (warp == 0) {
    best = warp_best[lane & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      const unsigned long long b = __shfl_xor_sync(0xffffffffu, best, o);
      best = b > best ? b : best;
    }
  }
  cluster.barrier_wait();   // all CTAs run: their memory can be written
  if (warp == 0 && lane < ctas) {
    Pub *const to = cluster.map_shared_rank(&mine, lane);
    to->told[rank].best = best;
    if (rank == 0) to->params = par;
  }
  cluster.sync();
  best = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) best = mine.told[c].best > best ? mine.told[c].best : best;
  const float temperature = mine.params.temperature, min_p = mine.params.min_p, u = mine.params.u;
  const float top_p = kTopP && mine.params.top_p < 1.0f ? mine.params.top_p : 1.0f;   // NaN: off
  const int32_t top_k = mine.params.top_k;
  const uint32_t top_key = static_cast<uint32_t>(best >> 32);

  // rows without a choice
  const bool live = mine.params.live != 0;
  if (!live || top_key <= kKeyMasked || !(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f) {
    if (live && rank == 0 && tid == 0) {
      const bool empty = top_key <= kKeyMasked;
      a.token[row] = empty ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(best));
      if (a.logprob != nullptr) a.logprob[row] = empty ? -INFINITY : 0.0f;
    }
    return;   // nobody reads or writes another CTA's memory any more
  }

  Row local;   // in registers, for the loops over the row
  local.top = radix_key_value(top_key);
  if (local.top == INFINITY) {   // those at +inf alone have a weight, the same
    local.top = 0.0f;
    for (int t = lane; t < len; t += 32) own[t] = Q::one(own[t]) == INFINITY ? static_cast<T>(0) : Q::masked();
    __syncwarp();
  }
  local.temperature = fminf(fmaxf(temperature, 0x1p-60f), 0x1p60f);
  local.c_hi = mine.params.c_hi;
  local.c_lo = mine.params.c_lo;
  local.ref = fabsf(local.top * local.c_hi) <= 128.0f ? 0.0f : local.top;
  {
    uint64_t minus, lo;
    exponents(local.top, local.top, local, minus, lo);
    local.whole_bits = (static_cast<uint32_t>(to_64ths(minus)) + 63u) & ~63u;
  }
  local.least = 1;
  if (tid == 0) r = local;   // for what is not inlined
  __syncthreads();
  if (min_p > 0.0f) {
    const uint64_t f = static_cast<uint64_t>(fminf(min_p, 1.0f) * 0x1p63f), w = weight(r.top, r, table);
    const uint64_t hi = __umul64hi(f, w), lo = f * w;
    local.least = (hi << 1 | lo >> 63) + (lo << 1 != 0 || f == 0 ? 1 : 0);
    if (tid == 0) r.least = local.least;
  }

  // f(tile, x[4]) over this warp's elements
  const auto each_tile = [&](auto f) {
#pragma unroll 1
    for (int t = 0; t < len; t += kTile) {
      float x[4];
      Q::get(*reinterpret_cast<const Vec *>(own + t + 4 * lane), x);
      f(t, x);
    }
  };
  // the same, two steps at a time
  const auto each_two_tiles = [&](auto f) {
    int t = 0;
#pragma unroll 1
    for (; t + kTile < len; t += 2 * kTile) {
      float x[4], y[4];
      Q::get(*reinterpret_cast<const Vec *>(own + t + 4 * lane), x);
      Q::get(*reinterpret_cast<const Vec *>(own + t + kTile + 4 * lane), y);
      f(t, x);
      f(t + kTile, y);
    }
    if (t < len) {
      float x[4];
      Q::get(*reinterpret_cast<const Vec *>(own + t + 4 * lane), x);
      f(t, x);
    }
  };
  // The sum of f(x, w, d) over the warp's elements with near(x, place).  Steps of a warp hold a few
  // of them, so a lane marks its own of 16 steps and then takes them two at a time: as many
  // weights as the lane with the most has, not as many as there are elements.
  const auto sum_of_some = [&](auto near, auto f) {
    uint64_t sum = 0;
#pragma unroll 1
    for (int t0 = 0; t0 < len; t0 += 16 * kTile) {
      uint32_t mask[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        mask[half] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = t0 + (8 * half + j) * kTile;
          if (t >= len) break;
          float x[4];
          Q::get(*reinterpret_cast<const Vec *>(own + t + 4 * lane), x);
#pragma unroll
          for (int k = 0; k < 4; ++k) mask[half] |= static_cast<uint32_t>(near(x[k], t + 4 * lane + k)) << (4 * j + k);
        }
      }
#pragma unroll 1
      while (__any_sync(0xffffffffu, (mask[0] | mask[1]) != 0)) {
        float x[2];
        bool here[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          here[i] = (mask[0] | mask[1]) != 0;
          const bool second = mask[0] == 0;
          const int b = max(__ffs(second ? mask[1] : mask[0]) - 1, 0);
          x[i] = Q::one(own[t0 + (b >> 2) * kTile + 4 * lane + (b & 3) + (second && here[i] ? 8 * kTile : 0)]);
          if (second) mask[1] &= mask[1] - 1;
          mask[0] &= mask[0] - 1;
        }
        Weights v;
        weights(x[0], x[1], local, table, v);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (here[i] && v.d[i] < kCut) sum += f(x[i], v.w[i], v.d[i]);
      }
    }
    return warp_total(sum);
  };
  // the warp's kept weights
  const auto kept_sums = [&](uint64_t threshold) {
    const auto kept = [&](uint64_t w) { return w >= local.least ? w : 0; };
    if (!(kTopK || kTopP) || threshold == 0) {
      uint64_t sum = 0;
      const auto all = [&](auto keep) {
        each_two_tiles([&](int, const float (&x)[4]) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            Weights v;
            weights(x[2 * h], x[2 * h + 1], local, table, v);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (v.d[i] < kCut) sum += keep(v.w[i]);
          }
        });
      };
      if (local.least == 1) all([](uint64_t w) { return w; });
      else all(kept);
      return warp_total(sum);
    }
    const float least_x = radix_key_value(static_cast<uint32_t>(threshold >> kIndexBits));
    const int last = (1 << kIndexBits) - 1 - static_cast<int>(threshold & ((1u << kIndexBits) - 1)) - begin;   // of its equals
    return sum_of_some([&](float x, int place) { return x > least_x || (x == least_x && place <= last); },
                       [&](float, uint64_t w, uint32_t) { return kept(w); });
  };
  // Those of the elements above a bin of exponents, or above part `fine` of it.
  const auto low_edge = [&](int32_t border) {   // less ref, a little lower
    return (__uint_as_float(local.whole_bits - static_cast<uint32_t>(border - 63)) - kMagic - 0x1.2p-7f) / local.c_hi;
  };
  const auto sum_above = [&](int32_t border, int32_t fine, uint64_t &all, uint64_t &kept) {   // and what min-p keeps of them
    const float least_x = low_edge(border);
    uint64_t small = 0;
    all = sum_of_some([&](float x, int) { return x - local.ref >= least_x; },
                      [&](float x, uint64_t w, uint32_t d) {
                        int32_t code = exponent_bin(d), at = border;
                        if (fine >= 0) {
                          uint64_t minus, lo;
                          exponents(x, x, local, minus, lo);
                          code = fine_code(minus, to_64ths(minus), d, 0);
                          at = border * kFine + fine;
                        }
                        if (code >= at) return static_cast<uint64_t>(0);
                        if (w < local.least) small += w;
                        return w;
                      });
    kept = all - (local.least > 1 ? warp_total(small) : 0);
  };
  const uint64_t f_u = u > 0.0f ? static_cast<uint64_t>(fminf(u, 0x1.fffffep-1f) * 0x1p64f) : 0ull;   // (NaN: 0)
  uint64_t threshold = 0;   // composite of the last kept element

  // top-k's border, then top-p's among what top-k keeps
  if constexpr (kTopK || kTopP)
  for (int kind = kTopK && top_k > 0 && top_k < a.p.V ? 0 : 1; kind < (kTopP && top_p < 1.0f ? 2 : 1); ++kind) {
    const bool mass = kTopP && (!kTopK || kind == 1);
    const uint64_t low = kTopK ? threshold : 0;   // top-p's elements are those >= low
    const auto among = [&](uint64_t c) { return !kTopK || c >= low; };
    uint64_t sum = 0;
    // leading bits of a weight in a word of the histogram, as many as this CTA's elements leave room for;
    // the last one always set, so that what is cut off has no direction
    const int lead = __clz(kWarps * len);
    if (mass) {
      each_two_tiles([&](int t, const float (&x)[4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          Weights v;
          weights(x[2 * h], x[2 * h + 1], local, table, v);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (v.d[i] < kCut && (!kTopK || low == 0 || among(composite(x[2 * h + i], begin + t + 4 * lane + 2 * h + i)))) {
              sum += v.w[i];
              atomicAdd(&hist[v.d[i] + 63], static_cast<uint32_t>(v.m[i] >> 32) >> (31 - lead) | 1u);
            }
          }
        }
      });
      sum = warp_total(sum);
      if (lane == 0) warp_above[warp] = sum;
    } else {
      each_two_tiles([&](int, const float (&x)[4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint64_t minus, lo;
          uint32_t d[2];
          exponents(x[2 * h], x[2 * h + 1], local, minus, lo);
          steps(to_64ths(minus), local, d);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (d[i] < kCut) atomicAdd(&hist[d[i] + 63], 1u);
        }
      });
    }
    push_octaves(hist, mine.octave);
    if (mass && warp == 0) {
      sum = warps_total(warp_above);
      if (lane < ctas) cluster.map_shared_rank(&mine, lane)->told[rank].all = sum;
    }
    cluster.sync();
    uint64_t want = static_cast<uint64_t>(top_k);
    if (mass) {
      uint64_t z = 0;
#pragma unroll
      for (int c = 0; c < kCtas; ++c) z += mine.told[c].all;
      want = ceil_product(top_p, z);
    }
    const float want_units = mass ? static_cast<float>(want) * __uint_as_float(static_cast<uint32_t>(127 + lead - 45) << 23) : static_cast<float>(want);
    const Exponent ex = find_exponent(mass, hist, mine.octave, s.bin, want_units);
    int32_t border = ex.bin;
    if (!mass && ex.all <= static_cast<float>(want)) {   // all that have a weight are kept
      cluster.sync();               // nobody reads the histogram any more
      clear_hist(hist, kYBins);
      __syncthreads();
      continue;
    }

    // Candidates in order of their index, and exactly what lies above them: of the border's
    // bin, or of its part `fine`; in the first round for top-k all from the top.  Where the leading
    // bits of the weights had missed the bin (a border very near its edge), again with its neighbour.
    bool listed = false;
    for (int misses = 0;; ++misses) {
      int32_t fine = -1, n = 0;
      bool from_top = false, empty = false, by_warp = false;   // by_warp: warp_kept is each warp's
      int32_t candidates = 0;   // of this warp
      uint64_t over = 0;   // what lies above the candidates in all CTAs
      ushort4 counts{};    // candidates of warps 4 * lane to 4 * lane + 3
      for (int round = 0; round < 2; ++round) {
        from_top = !mass && round == 0;
        uint64_t above = 0, kept = 0;
        // what this CTA has above, from its histogram: counts, and weights in the second round
        if (round == 1) {
          const int b = kBins - 1 - tid;
          if (b > kBins - 1 - fine) above = (mass ? static_cast<uint64_t>(hist[kBins + b]) << 32 : 0) + hist[b];
          if (tid == 0) above += mine.told[rank].above;
        } else if (!mass) {
#pragma unroll
          for (int k = 0; k < kYBins / kThreads; ++k) above += tid + k * kThreads < border ? hist[tid + k * kThreads] : 0;
        }
        const int32_t at_border = round == 0 ? border : border * kFine + fine;
        n = 0;
        // the border's bin as a range of logits less ref, a little wide: most steps of a warp hold none of it
        const float p_high = __uint_as_float(r.whole_bits - static_cast<uint32_t>(max(border - 63, 0))) - kMagic + 0x1.2p-7f;
        const float x_low = low_edge(border), x_high = from_top ? INFINITY : p_high / r.c_hi;
        each_tile([&](int t, const float (&x)[4]) {
          bool near = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) near = near || (x[k] - local.ref >= x_low && x[k] - local.ref <= x_high);
          if (!__any_sync(0xffffffffu, near)) return;
          int32_t code[4];   // the bin, and its part in the second round: smaller above
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint64_t minus, lo;
            uint32_t d[2];
            exponents(x[2 * h], x[2 * h + 1], local, minus, lo);
            const uint64_t t64 = to_64ths(minus);
            steps(t64, local, d);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              code[2 * h + i] = exponent_bin(d[i]);
              if (round == 1) code[2 * h + i] = fine_code(minus, t64, d[i], i);
            }
          }
          uint32_t take = 0;   // places among those taken: four ballots, a lane's elements side by side
          int32_t at = n;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool in = from_top ? code[k] <= at_border : code[k] == at_border;
            const uint32_t lanes = __ballot_sync(0xffffffffu, in);
            take |= static_cast<uint32_t>(in) << k;
            at += __popc(lanes & ((1u << lane) - 1));
            n += __popc(lanes);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (take >> k & 1) {
              if (at < Pub::kSegment) {
                mine.logit[warp][at] = own[t + 4 * lane + k];
                mine.place[warp][at] = static_cast<uint16_t>(t + 4 * lane + k);
              }
              ++at;
            }
          }
        });
        candidates = n;
        by_warp = mass && (round == 0 || local.least > 1);
        if (by_warp) sum_above(border, fine, above, kept);
        else above = kept = warp_total(above);
        if (lane == 0) {
          warp_above[warp] = above;
          warp_kept[warp] = kept;
        }
        if (lane < ctas) cluster.map_shared_rank(&mine, lane)->count[rank * kWarps + warp] = static_cast<uint16_t>(n);   // at most the range
        __syncthreads();
        if (warp == 0) {
          above = warps_total(warp_above);
          kept = warps_total(warp_kept);
          if (lane < ctas) {
            Pub *const to = cluster.map_shared_rank(&mine, lane);
            to->told[rank].above = above;
            to->told[rank].kept = kept;
          }
        }
        cluster.sync();

        // the list's length (every warp by itself), and what lies above it
        static_assert(kRanges == 128, "four counts a lane");
        counts = reinterpret_cast<const ushort4 *>(mine.count)[lane];
        n = __reduce_add_sync(0xffffffffu, counts.x + counts.y + counts.z + counts.w);
        const bool fits = __all_sync(0xffffffffu, max(max(counts.x, counts.y), max(counts.z, counts.w)) <= Pub::kSegment);
        over = 0;
#pragma unroll
        for (int c = 0; c < kCtas; ++c) over += mine.told[c].above;
        listed = n > 0 && n <= kListMost && fits;
        empty = n == 0;
        if (from_top && listed) over = 0;   // they are in the list themselves
        if (listed || round == 1 || over >= want || (mass && empty)) break;

        // too many: the bin's parts
        clear_hist(hist, 3 * kBins);
        __syncthreads();
        each_tile([&](int t, const float (&x)[4]) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint64_t minus, lo;
            uint32_t d[2];
            exponents(x[2 * h], x[2 * h + 1], local, minus, lo);
            const uint64_t t64 = to_64ths(minus);
            steps(t64, local, d);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (exponent_bin(d[i]) != border) continue;
              if (kTopK && low != 0 && !among(composite(x[2 * h + i], begin + t + 4 * lane + 2 * h + i))) continue;
              const uint32_t bin = kBins - 1 - fine_code(minus, t64, d[i], i) % kFine;
              if (mass) add_to_hist(hist, bin, weight(x[2 * h + i], r, table));
              else atomicAdd(&hist[bin], 1u);
            }
          }
        });
        cluster.sync();
        const Found f = find_bin(mass, ctas, hist, s, want - over);
        if (f.bin == kBins) break;   // the leading bits had missed the bin
        fine = kBins - 1 - static_cast<int32_t>(f.bin);
      }

      // the list: gathered and searched by the first CTA
      Verdict verdict{0, 0, 0, -1};
      if (listed && rank == 0) {
        if (warp == 0) {
          const int32_t four = counts.x + counts.y + counts.z + counts.w;
          int32_t at = four;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int32_t up = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += up;
          }
          at -= four;
          list_at[4 * lane] = at;
          list_at[4 * lane + 1] = at += counts.x;
          list_at[4 * lane + 2] = at += counts.y;
          list_at[4 * lane + 3] = at += counts.z;
          if (lane == 31) list_at[kRanges] = at + counts.w;
        }
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
          int w = 0;
#pragma unroll
          for (int step = kRanges / 2; step > 0; step >>= 1)
            if (list_at[w + step] <= i) w += step;
          const Pub *const from = cluster.map_shared_rank(&mine, w / kWarps);
          const int k = i - list_at[w];
          list[i] = composite(Q::one(from->logit[w % kWarps][k]), w * len + from->place[w % kWarps][k]);
        }
        if (from_top) cluster.barrier_arrive();   // everything that is kept is in the list: the other CTAs may go
        __syncthreads();
        const auto list_weight = [&](int i) { return weight(radix_key_value(static_cast<uint32_t>(list[i] >> kIndexBits)), r, table); };
        const auto kept_weight = [&](int i) {   // behind the search
          const uint64_t v = list[i] >= threshold ? list_weight(i) : 0;
          return v >= local.least ? v : 0;
        };
        const auto finish_listed = [&](uint64_t c, uint64_t total) {
          finish(a, row, (1 << kIndexBits) - 1 - static_cast<int>(c & ((1u << kIndexBits) - 1)), radix_key_value(static_cast<uint32_t>(c >> kIndexBits)),
                 total, r, table);
        };
        uint64_t *const part = reinterpret_cast<uint64_t *>(hist);   // [kThreads]
        bool found = true;
        // threads of an element of a small list; of others a thread has kChunk
        const int split = n <= 128 ? 4 : n <= kSmallList ? 2 : 0;
        uint64_t before = 0, list_total = 0, own_kept = 0;   // kept weights: before this thread's, all, its own
        if (n <= kSmallList) {
          // threads e * split .. for element e: its rank and the weight of what lies above it by looking at all
          ulonglong2 *const both = reinterpret_cast<ulonglong2 *>(hist);
          const int e = tid / split, part_of = tid % split;
          const bool here = e < n;
          const uint64_t mine_c = here ? list[e] : 0;
          if (tid < n) both[tid] = make_ulonglong2(list[tid], among(list[tid]) ? list_weight(tid) : 0);
          __syncthreads();
          const uint64_t mine_w = here ? both[e].y : 0;
          uint64_t higher = 0;
          uint32_t higher_n = 0;
          if (__any_sync(0xffffffffu, here)) {
#pragma unroll 4
            for (int j = part_of; j < n; j += split) {
              const ulonglong2 o = both[j];
              const bool above = o.x > mine_c;
              higher_n += above;
              higher += above ? o.y : 0;
            }
            for (int o = 1; o < split; o <<= 1) {
              higher_n += __shfl_xor_sync(0xffffffffu, higher_n, o);
              higher += __shfl_xor_sync(0xffffffffu, higher, o);
            }
          }
          bool keep = here && part_of == 0 && among(mine_c);
          if (!mass) keep = keep && over + higher_n < want;
          if (mass || (kTopP && from_top && top_p < 1.0f)) {
            const uint64_t some = warp_total(keep ? mine_w : 0);
            if (lane == 0) s.warp_sum[warp] = some;
            __syncthreads();
            const uint64_t all = warps_total(s.warp_sum);
            __syncthreads();
            if (mass) found = over < want && want <= over + all;
            keep = keep && (mass ? over + higher < want : higher < ceil_product(top_p, all));
          }
          // kept weights by place, behind `both`
          static_assert(kSmallList * (sizeof(ulonglong2) + sizeof(uint64_t)) <= kListOffset, "beside the list");
          uint64_t *const kept = reinterpret_cast<uint64_t *>(both + kSmallList);
          if (here && part_of == 0) kept[e] = keep && mine_w >= local.least ? mine_w : 0;
          const int kept_n = __syncthreads_count(keep);
          if (keep && higher_n == static_cast<uint32_t>(kept_n) - 1) s.composite = mine_c;
          __syncthreads();
          threshold = s.composite;
          if (warp == 0) {   // the rest is one warp's, which waits for nobody: up to eight a lane
            const int each = (n + 31) / 32, first = min(lane * each, n), last = min(first + each, n);
            for (int i = first; i < last; ++i) own_kept += kept[i];
            before = own_kept;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const uint64_t up = __shfl_up_sync(0xffffffffu, before, o);
              if (lane >= o) before += up;
            }
            list_total = __shfl_sync(0xffffffffu, before, 31);
            before -= own_kept;
            if (from_top) {
              const uint64_t at = __umul64hi(f_u, list_total);
              if (at >= before && at < before + own_kept) {
                int i = first;
                for (; at >= before + kept[i]; ++i) before += kept[i];
                finish_listed(list[i], list_total);
              }
            } else {   // sums before each
              for (int i = first; i < last; ++i) {
                const uint64_t w = kept[i];
                kept[i] = before;
                before += w;
              }
              __syncwarp();
              if (lane <= ctas) {
                const int i = list_at[lane * kWarps];
                cta_at[lane] = i < n ? kept[i] : list_total;
              }
            }
          }
        } else {
          const auto list_mass = [&](uint64_t from) {
            uint64_t v = 0;
            for (int i = tid; i < n; i += kThreads) v += list[i] >= from ? list_weight(i) : 0;
            const uint64_t all = exclusive_sum(v, s.warp_sum).all;
            __syncthreads();
            return all;
          };
          if (!mass) {
            threshold = descend_list(false, list, n, 0, want - over, r, table, hist, s);
            if (from_top && top_p < 1.0f) {
              const uint64_t z = list_mass(threshold);
              threshold = descend_list(true, list, n, threshold, ceil_product(top_p, z), r, table, hist, s);
            }
          } else {
            // the leading bits of the weights may have missed the bin
            found = over < want && want <= over + list_mass(low);
            if (found) threshold = descend_list(true, list, n, low, want - over, r, table, hist, s);
          }
          if (found && (mass || from_top)) {
#pragma unroll 1
            for (int i = tid * kChunk; i < min((tid + 1) * kChunk, n); ++i) own_kept += kept_weight(i);
            const Sums kept_sums = exclusive_sum(own_kept, s.warp_sum);
            before = kept_sums.before;
            list_total = kept_sums.all;
            part[tid] = before;
          }
        }
        if (from_top) {
          const uint64_t at = __umul64hi(f_u, list_total);
          if (n > kSmallList && at >= before && at < before + own_kept) {
            int i = tid * kChunk;
            for (uint64_t v; at >= before + (v = kept_weight(i)); ++i) before += v;
            finish_listed(list[i], list_total);
          }
          cluster.barrier_wait();
          return;
        }
        verdict.threshold = threshold;
        if (mass && found && n > kSmallList) {
          // up to each CTA's part: the list's kept weights before it
          __syncthreads();
          if (tid <= ctas) {
            const int i = list_at[tid * kWarps], t = i / kChunk;   // the thread that has it
            uint64_t at = t < kThreads ? part[t] : list_total;
#pragma unroll 1
            for (int j = t * kChunk; j < i; ++j) at += kept_weight(j);
            cta_at[tid] = at;
          }
        }
        if (mass && found && warp == 0) {
          __syncwarp();
          // the CTA in which the sums pass u Z
          const int c = lane & (kCtas - 1);
          const uint64_t here = c < ctas ? mine.told[c].kept + cta_at[c + 1] - cta_at[c] : 0;
          uint64_t upto = here;
#pragma unroll
          for (int o = 1; o < kCtas; o <<= 1) {
            const uint64_t up = __shfl_up_sync(0xffffffffu, upto, o, kCtas);
            if (c >= o) upto += up;
          }
          verdict.total = __shfl_sync(0xffffffffu, upto, kCtas - 1);
          const uint64_t at = __umul64hi(f_u, verdict.total);
          verdict.owner = __ffs(__ballot_sync(0xffffffffu, at < upto)) - 1;
          verdict.at = at - __shfl_sync(0xffffffffu, upto - here, verdict.owner);
        } else if (!mass) {
          verdict.owner = 0;
        }
        if (warp == 0 && lane < ctas) cluster.map_shared_rank(&mine, lane)->verdict = verdict;
      } else if (listed && from_top) {
        cluster.sync();
        return;
      }
      if (listed) {
        cluster.sync();
        verdict = mine.verdict;
        threshold = verdict.threshold;
        listed = verdict.owner >= 0;
        if (mass && listed) {
          if (rank == verdict.owner) {
            // its warps' kept weights: what lies above the border, and of the candidates
            uint64_t kept = 0;
            if (by_warp) {
              for (int i = lane; i < candidates; i += 32) {
                const float x = Q::one(mine.logit[warp][i]);
                if (composite(x, begin + mine.place[warp][i]) < threshold) continue;
                const uint64_t w = weight(x, r, table);
                if (w >= local.least) kept += w;
              }
              kept = warp_total(kept) + warp_kept[warp];
              __syncwarp();
            } else {
              kept = kept_sums(threshold);
            }
            if (lane == 0) warp_kept[warp] = kept;
            __syncthreads();
            pick<T>(a, row, data, rank, warp_kept, 0, verdict.at, threshold, verdict.total, r, table, tile_sum);
          }
          return;
        }
      } else if (mass && (empty || over >= want)) {
        cluster.sync();   // nobody reads these counts any more
      } else {
        break;
      }
      if (listed || !mass || misses == 2) break;
      border += over >= want ? -1 : 1;
      if (border < 0 || border >= kYBins) break;
    }
    if (!listed) {
      // long lists: a descent over the row
      uint64_t left = want, prefix = 0;
      for (int shift = kCompositeBits; shift > 0;) {
        const int known = shift, bits = min(kDigit, shift);
        shift -= bits;
        cluster.sync();   // nobody reads the histogram any more
        clear_hist(hist, 3 * kBins);
        __syncthreads();
        each_tile([&](int t, const float (&x)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t c = composite(x[k], begin + t + 4 * lane + k);
            if (key_of(x[k]) <= kKeyMasked || !among(c) || c >> known != prefix) continue;
            const uint32_t at = static_cast<uint32_t>(c >> shift) & ((1u << bits) - 1);
            if (!mass) atomicAdd(&hist[at], 1u);
            else if (const uint64_t v = weight(x[k], r, table); v != 0) add_to_hist(hist, at, v);
          }
        });
        cluster.sync();
        const Found f = find_bin(mass, ctas, hist, s, left);
        prefix = prefix << bits | f.bin;
        left -= f.above;
      }
      threshold = prefix;
    }
    cluster.sync();   // nobody reads what is written next
    clear_hist(hist, kYBins);
    __syncthreads();
  }

  // the kept weights of the row
  uint64_t sum = kept_sums(threshold);
  if (lane == 0) warp_kept[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    sum = warps_total(warp_kept);
    if (lane < ctas) cluster.map_shared_rank(&mine, lane)->told[rank].sum = sum;
  }
  cluster.sync();
  uint64_t total = 0, reach = 0, here = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    const uint64_t v = mine.told[c].sum;
    if (c < rank) reach += v;
    if (c == rank) here = v;
    total += v;
  }
  const uint64_t at = __umul64hi(f_u, total);
  if (at >= reach && at < reach + here)
    pick<T>(a, row, data, rank, warp_kept, reach, at, threshold, total, r, table, tile_sum);
}

// Clusters of 1, 2, 4 and 8 CTAs that run at a time: two CTAs to an SM, and one.
struct Room {
  int clusters[2][4];
};
template <typename T, bool kTopK, bool kTopP>
cudaError_t launch(SampleArgs a, cudaStream_t stream) {
  constexpr bool kList = kTopK || kTopP;
  constexpr int kFixed = static_cast<int>(fixed_smem<T, kList>());
  // dynamic shared memory with two CTAs to an SM, and that leaves room for one
  constexpr int kHalf = 112 * 1024 - static_cast<int>(sizeof(Shared<T, kList>)) - 11 * 1024, kAlone = 120 * 1024;
  constexpr int kMost = std::max(kAlone, kFixed + IDX_MAX_VOCAB / kCtas * static_cast<int>(sizeof(T)));
  static std::mutex mu;
  static bool done[128];
  static Room rooms[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once_per_device(mu, done, [dev] {
    cudaError_t got = cudaFuncSetAttribute(sample_kernel<T, kTopK, kTopP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    for (int alone = 0; alone < 2; ++alone) {
      for (int k = 0; k < 4 && got == cudaSuccess; ++k) {
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 1u << k;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(1u << k);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(alone ? kAlone : kHalf);
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        got = cudaOccupancyMaxActiveClusters(&rooms[dev].clusters[alone][k], sample_kernel<T, kTopK, kTopP>, &cfg);
      }
    }
    return got;
  });
  if (e != cudaSuccess) return e;

  // CTAs of a row, and whether an SM has one or two of them: by the cycles that all rows take in
  // waves of the clusters that fit.  A CTA takes about 15,000 and one a logit beside another one,
  // seven tenths of that alone (64 x 128,000 bf16: four in pairs 22.9 us where eight took 27.7; 8 x 151,552
  // fp32: eight alone 14.9 us, in pairs, which the hardware takes where they fit, 16.9).
  int64_t best = 0;
  int smem = 0;
  a.ctas = 0;
  for (int k = 3; k >= 0; --k) {
    const int ctas = 1 << k, len = (a.p.V + ctas * kWarps * kTile - 1) / (ctas * kWarps * kTile) * kTile;
    const int need = kFixed + kWarps * len * static_cast<int>(sizeof(T));
    if (len > 2 * kWarps * kTile || need > kMost) break;
    for (int alone = 0; alone < 2; ++alone) {
      const int64_t fit = rooms[dev].clusters[alone][k];
      if (fit < 1 || (alone == 0 && need > kHalf)) continue;
      const int64_t cycles = (a.p.R + fit - 1) / fit * (15000 + a.p.V / ctas) * (alone ? 7 : 10);
      if (a.ctas == 0 || cycles < best) {
        best = cycles;
        a.ctas = ctas;
        a.warp_len = len;
        smem = alone ? std::max(need, kAlone) : need;
      }
    }
  }
  if (a.ctas == 0) return cudaErrorInvalidConfiguration;
  return launch_early(sample_kernel<T, kTopK, kTopP>, static_cast<unsigned>(a.p.R) * static_cast<unsigned>(a.ctas), kThreads,
                      static_cast<size_t>(smem), static_cast<unsigned>(a.ctas), stream, a);
}

template <typename T>
cudaError_t launch(const SampleArgs &a, cudaStream_t stream) {
  constexpr int kSpan = kCtas * kWarps * kTile;
  static_assert(IDX_MAX_VOCAB % kSpan == 0 && IDX_MAX_VOCAB / kRanges / kTile <= 2 * kWarps, "whole steps of every warp");
  if (a.p.top_k != nullptr) return a.p.top_p != nullptr ? launch<T, true, true>(a, stream) : launch<T, true, false>(a, stream);
  return a.p.top_p != nullptr ? launch<T, false, true>(a, stream) : launch<T, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
  return a.p.logits_dtype == IDX_LOGITS_F32 ? launch<float>(a, stream) : launch<uint16_t>(a, stream);
}

}  // namespace idx
