// A token of every row of logits: temperature, top-k, top-p and min-p, drawn with given
// random numbers.
//
// Eight CTAs, a cluster, hold one row in shared memory: the logits are read once, and what
// the CTAs need of each other (maxima, histograms, sums) they read from each other's shared
// memory between cluster barriers.  Every CTA then finds the same thresholds from the same
// numbers; parameters come from the first CTA's copy, so that no barrier depends on memory
// that could change in between.
//
// A token may not depend on how sums are rounded, and a border (u Z between two tokens' sums,
// p Z between two masses) lies within 2^-24 of some sum in a percent of the rows.  So weights
// are integers: w = 2^43 exp((l - max l) / T), off by about 2^-39 of itself or half a unit,
// their sums are exact in 64 bits whatever the order, and the comparisons with p Z and u Z
// exact in 128.
//
// Thresholds: the kept tokens are a prefix of the order (logit descending, index ascending),
// ending at a key (the logit's order-preserving 32 bits) of whose equals the first `ties` by
// index are kept.  Both top-k and top-p find it by radix descent, 11, 11 and 10 bits, over
// histograms of counts and of weights.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <mutex>

#include "idx_device.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace idx {
namespace {

constexpr int kCtas = 8;         // of a cluster: a row
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 128;       // a warp's step: four elements a lane
constexpr int kBins = 2048;
constexpr uint32_t kKeyMasked = 0x007FFFFFu;   // radix_key(-inf)
constexpr int kOneBits = 43;
constexpr uint64_t kOne = 1ull << kOneBits;    // the largest logit's weight

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

// A row's parameters and what follows from its largest logit.
struct Row {
  float top;          // the largest logit
  float temperature;  // within 2^-60 .. 2^60
  float c_hi, c_lo;   // log2(e) / T in two terms
};

// 2^43 exp((x - top) / T), rounded: with y = (top - x) log2(e) / T in two terms, 2^-y is a
// power of two, a table entry of 8 bits and exp(g) - 1 of the rest g, |g| <= 2^-9.5, whose
// leading term is kept apart so that integers hold it to 2^-40.
__device__ __forceinline__ uint64_t weight(float x, const Row &r, const uint64_t *exp2_table) {
  constexpr float kMagic = 49152.0f;   // 1.5 * 2^15: a sum's last bit is 1 / 256
  constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
  // top - x = s + e exactly (Knuth's sum of two terms)
  const float s = r.top - x, b = s - r.top, e = (r.top - (s - b)) - (x + b);
  const float y = s * r.c_hi;
  float yl = fmaf(s, r.c_hi, -y);
  yl = fmaf(s, r.c_lo, yl);
  yl = fmaf(e, r.c_hi, yl);
  const float t = y + kMagic;
  const int ti = __float_as_int(t) - __float_as_int(kMagic);   // y in units of 1 / 256
  const float f = (t - kMagic) - y;                            // 2^-y = 2^(-ti / 256) 2^(f - yl)
  const float h = f * kLn2Hi;
  float hl = fmaf(f, kLn2Hi, -h);
  hl = fmaf(f, kLn2Lo, hl);
  hl = fmaf(-yl, kLn2Hi, hl);
  const float q = fmaf(h, fmaf(h, fmaf(h, 1.0f / 6.0f, 0.5f), hl), hl);
  const int g = __float2int_rn(h * 0x1p40f) + __float2int_rn(q * 0x1p40f);
  const uint64_t p = exp2_table[-ti & 255];                    // 2^44 times 1 .. 2
  const int n = (ti + 255) >> 8;
  const uint64_t w2 = p + static_cast<uint64_t>((static_cast<int64_t>(static_cast<int32_t>(p >> 14)) * g) >> 26);
  const uint64_t w = ((w2 >> (n & 63)) + 1) >> 1;
  // the largest has weight 1 also where it is infinite; masked ones (and NaN) have none
  return x == r.top ? kOne : y < 43.9f ? w : 0ull;
}

// What the CTAs of a row publish, one struct per CTA; every field is written once.
struct Shared {
  // the first CTA's: the row's parameters
  float temperature, top_p, min_p, u;
  int32_t top_k, live;
  unsigned long long best;   // (key << 32) | ~index of the CTA's largest
  uint64_t sum_above;        // weights above the threshold
  uint32_t equals;           // elements at the threshold
};

template <typename T>
struct Quad;
template <>
struct Quad<float> {
  using Vec = float4;
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
  static __device__ __forceinline__ void get(const Vec &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ float one(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ uint16_t masked() { return 0xFF80u; }
};

__device__ __forceinline__ uint32_t key_of(float x) { return x != x ? kKeyMasked : radix_key(x); }

// The bin of a row's histogram, from the top, at which the running sum reaches `target`
// (1 .. the sum of all): bin, the sum above it and its own.  All threads of all CTAs call;
// `target` is a function of the sum of all.
struct Found {
  uint32_t bin;
  uint64_t above, own;
};
struct Scan {
  uint64_t warp_sum[kWarps];
  Found found;
};
template <bool kWide, typename F>
__device__ __forceinline__ Found find_bin(cg::cluster_group &cluster, uint32_t *hist, Scan &scan, F target) {
  constexpr int kPer = kBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t own[kPer] = {}, sum = 0;
  const int first = kBins - kPer * (tid + 1);   // this thread's bins, ascending
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    const uint32_t *const remote = cluster.map_shared_rank(hist, c);
    const uint4 lo = *reinterpret_cast<const uint4 *>(remote + first);
    own[0] += lo.x;
    own[1] += lo.y;
    own[2] += lo.z;
    own[3] += lo.w;
    if constexpr (kWide) {
      const uint4 hi = *reinterpret_cast<const uint4 *>(remote + kBins + first);
      own[0] += static_cast<uint64_t>(hi.x) << 32;
      own[1] += static_cast<uint64_t>(hi.y) << 32;
      own[2] += static_cast<uint64_t>(hi.z) << 32;
      own[3] += static_cast<uint64_t>(hi.w) << 32;
    }
  }
  static_assert(kPer == 4, "a thread's bins are one vector");
#pragma unroll
  for (int i = 0; i < kPer; ++i) sum += own[i];
  uint64_t upto = sum;   // bins from the top through this thread's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 31) scan.warp_sum[warp] = upto;
  __syncthreads();
  uint64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan.warp_sum[w];
    total += scan.warp_sum[w];
  }
  const uint64_t want = target(total);
  uint64_t above = before + upto - sum;
#pragma unroll
  for (int i = kPer - 1; i >= 0; --i) {
    if (above < want && want <= above + own[i]) scan.found = {static_cast<uint32_t>(first + i), above, own[i]};
    above += own[i];
  }
  __syncthreads();
  return scan.found;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  using Q = Quad<T>;
  using Vec = typename Q::Vec;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint32_t *const hist = reinterpret_cast<uint32_t *>(smem_raw);   // [2][low, high][kBins]
  T *const data = reinterpret_cast<T *>(smem_raw + 4 * kBins * sizeof(uint32_t));
  __shared__ Shared mine;
  __shared__ Scan scan;
  __shared__ uint64_t table[256];
  __shared__ unsigned long long warp_best[kWarps];
  __shared__ uint64_t warp_sum[kWarps];
  __shared__ uint32_t warp_equals[kWarps];

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / kCtas;
  // this warp's elements: [begin, begin + len) of the row, those past V masked
  const int len = a.warp_len;
  const int begin = (rank * kWarps + warp) * len;
  T *const own = data + warp * len;
  const T *const src = static_cast<const T *>(a.p.logits) + row * a.p.ld;

  for (int i = tid; i < 256; i += kThreads) table[i] = kExp2.v[i];
  for (int i = tid; i < 4 * kBins; i += kThreads) hist[i] = 0;
  if (rank == 0 && tid == 0) {
    mine.live = a.p.rows == nullptr || row < *a.p.rows;
    mine.temperature = a.p.temperature != nullptr ? a.p.temperature[row] : 1.0f;
    mine.top_k = a.p.top_k != nullptr ? a.p.top_k[row] : 0;
    mine.top_p = a.p.top_p != nullptr ? a.p.top_p[row] : 1.0f;
    mine.min_p = a.p.min_p != nullptr ? a.p.min_p[row] : 0.0f;
    mine.u = a.p.u[row];
  }

  // the row, once, and its largest element (the first of several)
  unsigned long long best = 0;
  for (int t = 0; t < len; t += kTile) {
    const int i = begin + t + 4 * lane;
    Vec v;
    T *const e = reinterpret_cast<T *>(&v);
    if (a.vec && i + 4 <= a.p.V) {
      v = __ldcs(reinterpret_cast<const Vec *>(src + i));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = i + k < a.p.V ? src[i + k] : Q::masked();
    }
    *reinterpret_cast<Vec *>(own + t + 4 * lane) = v;
    float x[4];
    Q::get(v, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned long long b = static_cast<unsigned long long>(key_of(x[k])) << 32 | static_cast<uint32_t>(~(i + k));
      best = b > best ? b : best;
    }
  }
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
  const Shared *const first = cluster.map_shared_rank(&mine, 0);
  const float temperature = first->temperature, top_p = first->top_p, min_p = first->min_p, u = first->u;
  const int32_t top_k = first->top_k;
  const bool live = first->live != 0;
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
  {
    r.temperature = fminf(fmaxf(temperature, 0x1p-60f), 0x1p60f);
    const double c = 1.4426950408889634 / static_cast<double>(r.temperature);
    r.c_hi = static_cast<float>(c);
    r.c_lo = static_cast<float>(c - static_cast<double>(r.c_hi));
  }

  // f(key, x, index) over this warp's elements, four at a time in index order
  const auto each = [&](auto f) {
    for (int t = 0; t < len; t += kTile) {
      float x[4];
      Q::get(*reinterpret_cast<const Vec *>(own + t + 4 * lane), x);
#pragma unroll
      for (int k = 0; k < 4; ++k) f(key_of(x[k]), x[k]);
    }
  };
  int level = 0;   // of both descents together: they take turns with two histograms
  const auto next_hist = [&]() { return hist + (level & 1) * 2 * kBins; };
  // after a barrier nobody reads the other histogram any more
  const auto clear_other = [&]() {
    ++level;
    uint32_t *const h = next_hist();
    for (int i = tid; i < 2 * kBins; i += kThreads) h[i] = 0;
  };

  uint32_t tau = kKeyMasked, ties = 0;   // kept: keys above tau, and the first `ties` equal to it
  uint64_t dropped = 0;                  // the weight of those equal to it that are not kept
  if (top_k > 0 && top_k < a.p.V) {
    uint64_t left = static_cast<uint64_t>(top_k), equals = 0;
    uint32_t prefix = 0;
    bool all = false;   // no more than k elements are not masked
#pragma unroll 1
    for (int shift = 21; !all; shift -= shift > 10 ? 11 : 10) {
      const int bits = shift == 0 ? 10 : 11, known = shift + bits;   // 32 at first
      uint32_t *const h = next_hist();
      each([&](uint32_t key, float) {
        if (key > kKeyMasked && (known == 32 || key >> known == prefix)) atomicAdd(&h[(key >> shift) & ((1u << bits) - 1)], 1u);
      });
      cluster.sync();
      const Found f = find_bin<false>(cluster, h, scan, [&](uint64_t total) {
        all = total <= left;
        return left;
      });
      clear_other();
      prefix = prefix << bits | f.bin;
      left -= f.above;
      equals = f.own;
      all = all && known == 32;
      __syncthreads();   // the cleared histogram
      if (shift == 0) break;
    }
    if (!all) {
      tau = prefix;
      ties = static_cast<uint32_t>(left);
      dropped = (equals - left) * weight(radix_key_value(tau), r, table);
    }
  }
  if (top_p < 1.0f) {
    const uint32_t lowest = ties > 0 ? tau : tau + 1;
    uint64_t left = 0, class_mass = 0;
    uint32_t prefix = 0;
#pragma unroll 1
    for (int shift = 21;; shift -= shift > 10 ? 11 : 10) {
      const int bits = shift == 0 ? 10 : 11, known = shift + bits;
      uint32_t *const h = next_hist();
      each([&](uint32_t key, float x) {
        if (key >= lowest && (known == 32 || key >> known == prefix)) {
          const uint64_t w = weight(x, r, table);
          if (w == 0) return;
          const uint32_t bin = (key >> shift) & ((1u << bits) - 1);
          const uint32_t lo = static_cast<uint32_t>(w), was = atomicAdd(&h[bin], lo);
          const uint32_t hi = static_cast<uint32_t>(w >> 32) + (was + lo < was ? 1u : 0u);
          if (hi != 0) atomicAdd(&h[kBins + bin], hi);
        }
      });
      cluster.sync();
      const Found f = find_bin<true>(cluster, h, scan, [&](uint64_t total) {
        // the masses before kept tokens are below p Z: as integers, below its ceiling
        if (known == 32) {
          const uint64_t z = total - dropped, p = static_cast<uint64_t>(top_p * 0x1p64f);
          left = __umul64hi(p, z) + (p == 0 || p * z != 0 ? 1 : 0);
        }
        return left;
      });
      clear_other();
      prefix = prefix << bits | f.bin;
      left -= f.above;
      class_mass = f.own;
      __syncthreads();
      if (shift == 0) break;
    }
    // of the elements at the threshold those with i w < left, i = 0, 1, ..; of top-k's own no more than it keeps
    const uint64_t w = weight(radix_key_value(prefix), r, table), n = min((left + w - 1) / w, class_mass / w);
    ties = static_cast<uint32_t>(prefix == tau && ties > 0 ? min(n, static_cast<uint64_t>(ties)) : n);
    tau = prefix;
  }
  const uint64_t tau_weight = ties > 0 ? weight(radix_key_value(tau), r, table) : 0;
  const uint64_t least = min_p > 0.0f ? static_cast<uint64_t>(ceil(static_cast<double>(fminf(min_p, 1.0f)) * static_cast<double>(kOne))) : 1;
  if (tau_weight < least) ties = 0;

  // the weights above the threshold and the elements at it
  uint64_t sum = 0;
  uint32_t equals = 0;
  each([&](uint32_t key, float x) {
    if (key > tau) {
      const uint64_t w = weight(x, r, table);
      if (w >= least) sum += w;
    } else if (key == tau) {
      ++equals;
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  equals = __reduce_add_sync(0xffffffffu, equals);
  if (lane == 0) {
    warp_sum[warp] = sum;
    warp_equals[warp] = equals;
  }
  __syncthreads();
  if (tid == 0) {
    uint64_t s = 0;
    uint32_t n = 0;
    for (int w = 0; w < kWarps; ++w) {
      s += warp_sum[w];
      n += warp_equals[w];
    }
    mine.sum_above = s;
    mine.equals = n;
  }
  cluster.sync();
  // every thread: the row's sum, this CTA's part of it
  uint64_t before = 0, total = 0, part = 0;
  uint32_t equals_before = 0, seen = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    const Shared *const s = cluster.map_shared_rank(&mine, c);
    const uint32_t n = s->equals, kept = min(n, ties - min(ties, seen));
    const uint64_t here = s->sum_above + kept * tau_weight;
    if (c < rank) before += here;
    if (c == rank) {
      part = here;
      equals_before = seen;
    }
    seen += n;
    total += here;
  }
  cluster.sync();   // nobody reads another CTA's memory from here on
  const float uc = u > 0.0f ? u : 0.0f;
  const uint64_t at = __umul64hi(uc < 1.0f ? static_cast<uint64_t>(uc * 0x1p64f) : ~0ull, total);   // floor(u Z)
  if (at < before || at >= before + part) return;

  // the warp, the step and the element in which the sums pass u Z
  uint64_t reach = before;
  int w_at = 0;
  for (int w = 0; w < kWarps; ++w) {
    const uint32_t kept = min(warp_equals[w], ties - min(ties, equals_before));
    const uint64_t here = warp_sum[w] + kept * tau_weight;
    w_at = w;
    if (at < reach + here) break;
    reach += here;
    equals_before += warp_equals[w];
  }
  if (warp != w_at) return;
  uint32_t allowed = ties - min(ties, equals_before);
  for (int t = 0; t < len; t += kTile) {
    float x[4];
    Q::get(*reinterpret_cast<const Vec *>(own + t + 4 * lane), x);
    uint32_t n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) n += key_of(x[k]) == tau;
    uint32_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    const uint32_t tile_equals = __shfl_sync(0xffffffffu, upto, 31);
    uint32_t mine_before = upto - n;
    uint64_t w[4], s = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t key = key_of(x[k]);
      w[k] = 0;
      if (key > tau) {
        w[k] = weight(x[k], r, table);
        if (w[k] < least) w[k] = 0;
      } else if (key == tau) {
        if (mine_before < allowed) w[k] = tau_weight;
        ++mine_before;
      }
      s += w[k];
    }
    uint64_t sums = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(0xffffffffu, sums, o);
      if (lane >= o) sums += up;
    }
    uint64_t from = reach + sums - s;
    if (at >= from && at < from + s) {   // one lane of one warp of one CTA
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (at >= from && at < from + w[k]) {
          a.token[row] = begin + t + 4 * lane + k;
          // log(w / Z) from the logit itself, whose weight may be a few units, and log1p of Z - 1
          if (a.logprob != nullptr) {
            const double y = x[k] == r.top ? 0.0 : (static_cast<double>(r.top) - static_cast<double>(x[k])) / r.temperature;
            const float z = static_cast<float>(static_cast<double>(total - kOne) * 0x1p-43);
            a.logprob[row] = 0.0f - static_cast<float>(y) - log1pf(z);
          }
        }
        from += w[k];
      }
    }
    reach += __shfl_sync(0xffffffffu, sums, 31);
    if (reach > at) return;
    allowed -= min(allowed, tile_equals);
  }
}

constexpr int kFixedSmem = 4 * kBins * sizeof(uint32_t);

template <typename T>
cudaError_t launch(SampleArgs a, cudaStream_t stream) {
  constexpr int kMost = kFixedSmem + IDX_MAX_VOCAB / kCtas * static_cast<int>(sizeof(T));
  static_assert(IDX_MAX_VOCAB % (kCtas * kWarps * kTile) == 0, "whole steps of every warp");
  static std::mutex mu;
  static bool done[128];
  cudaError_t e = once_per_device(mu, done, [] {
    return cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  });
  if (e != cudaSuccess) return e;
  constexpr int kSpan = kCtas * kWarps * kTile;
  a.warp_len = static_cast<int32_t>((a.p.V + kSpan - 1) / kSpan) * kTile;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {kCtas, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.p.R) * kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kFixedSmem + static_cast<size_t>(kWarps) * a.warp_len * sizeof(T);
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
