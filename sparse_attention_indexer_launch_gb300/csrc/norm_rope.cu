// Norms of queries and keys for each head, their rotation, and keys and values into the
// paged cache, in one pass over a projection's output.
//
// A vector of D values (one head of a row) is a group of D / 8 lanes with eight values each,
// four pairs that turn together, so that the rotation stays within a lane: two runs of four
// for halves, one of eight for interleaved pairs.  It is read once and written once.  A warp
// takes a row, or a part of one where there are few: its lanes keep the cosines and sines of
// their four pairs in registers, and go through batches of a few heads, first of q, then of
// k, then of v, with the next batch's copies on their way to a lane's own place in shared
// memory.  Warps share nothing, so no barrier holds them up; two values ride in an instruction.
//
// What bounds it: memory.  16,209 rows of 64 + 2 x 8 heads of 128 into an E4M3 cache take 103 us,
// 6.1 TB/s or 90% of the measured copy bandwidth; 8,855 rows of 16 + 2 x 16 heads turned by three axes,
// bf16, 37.3 us, 86%; 40,000 rows reach 98 to 100%, so what is missing is start and end.  28 warps to
// an SM with one head at a time: 24 with 80 registers took 115 us and 40.7, 32 with 64 spill (127; one
// head at a time 103.5).  Groups of rows to a CTA, angles in shared memory behind a barrier, took 113
// and 42.2, two heads at a time 107 and 37.7.  A few rows: 2.7 us in a graph, which is launch, one read
// and one write.  With LayerNorm the first case takes 126 us, 74% (20 warps to an SM with up to 96
// registers; keys alone with it 118); heads of 64, 128 and 256 without a cache, RMS norm, 16,209 rows,
// 93 to 96%.  One to three fills of the GPU lose more: 5,000 rows 66 to 88%.
//
// Angles: positions reach 2^31, where pos * inv_freq in fp32 is off by whole turns.  The
// frequency in turns, inv_freq / (2 pi), is a fixed-point fraction of 64 bits, and a
// product with an integer position wraps at whole turns by itself.
#include <algorithm>

#include "idx_device.cuh"
#include "kv_quant.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kVectors = 4;     // heads of a lane in a batch

// inv_freq / (2 pi) in units of 2^-64 turn, modulo one turn: the 24-bit significand times
// 2^64 / (2 pi), shifted by the exponent and rounded.  Off by half a unit and, as the constant is
// off by 0.497, by 0.497 |inv_freq|.
__device__ __forceinline__ uint64_t turns_per_position(float inv_freq) {
  constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;   // 2^64 / (2 pi)
  const uint32_t u = __float_as_uint(inv_freq);
  const uint32_t ex = (u >> 23) & 0xFFu;
  const uint64_t m = (u & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int down = 150 - static_cast<int>(ex ? ex : 1u);   // the value is m * 2^-down
  uint64_t f;
  if (down <= 0) f = -down < 64 ? lo << -down : 0ull;
  else if (down < 64) f = (lo >> down | hi << (64 - down)) + (lo >> (down - 1) & 1u);
  else if (down == 64) f = hi + (lo >> 63);
  else f = down < 128 ? ((hi >> (down - 65)) + 1u) >> 1 : 0ull;   // hi has 22 bits
  return u >> 31 ? 0ull - f : f;
}

__device__ __forceinline__ float2 cos_sin(int32_t pos, float inv_freq) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns_per_position(inv_freq);
  // the nearest quarter turn, and what is left of it, within an eighth: 32 of the 64 bits, rounded
  // (for 2^31 positions and |inv_freq| <= 1 off by 2^-32 of a turn in all), then fp32 at that smaller size
  const uint32_t turn = static_cast<uint32_t>((phase + 0x80000000ull) >> 32), quarter = (turn + 0x20000000u) >> 30;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(turn - (quarter << 30))) * 0x1p-31f, &s, &c);
  if (quarter & 1u) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2u) {
    c = -c;
    s = -s;
  }
  if (!(fabsf(inv_freq) <= 3.402823466e38f)) s = c = __int_as_float(0x7FFFFFFF);   // no angle
  return make_float2(c, s);
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int kLanes>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t both(float v) { return pack2(v, v); }
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t &>(p);
}
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Where a lane's four pairs lie in a head: elements a + k and b + k (halves, two runs; dimensions
// that do not turn come as pairs as well), or a + 2 k and a + 2 k + 1.
struct Place {
  int a, b;
  bool turns;
};
template <bool kInterleaved>
__device__ __forceinline__ Place place_of(int lane, int rot) {
  Place p;
  p.turns = 8 * lane < rot;
  p.a = kInterleaved || !p.turns ? 8 * lane : 4 * lane;
  p.b = kInterleaved ? p.a + 1 : p.turns ? rot / 2 + 4 * lane : p.a + 4;
  return p;
}

// Values of a lane's pairs, two in a word: a[0] holds those of a + 0 and a + 1 (of pairs 0 and 1).
struct Pairs {
  uint64_t a[2], b[2];
};
template <bool kInterleaved>
__device__ __forceinline__ Pairs unpack(const uint4 &v) {
  Pairs x;
  if constexpr (kInterleaved) {
    x.a[0] = pack2(bf16_low(v.x), bf16_low(v.y));
    x.b[0] = pack2(bf16_high(v.x), bf16_high(v.y));
    x.a[1] = pack2(bf16_low(v.z), bf16_low(v.w));
    x.b[1] = pack2(bf16_high(v.z), bf16_high(v.w));
  } else {
    x.a[0] = pack2(bf16_low(v.x), bf16_high(v.x));
    x.a[1] = pack2(bf16_low(v.y), bf16_high(v.y));
    x.b[0] = pack2(bf16_low(v.z), bf16_high(v.z));
    x.b[1] = pack2(bf16_low(v.w), bf16_high(v.w));
  }
  return x;
}
template <bool kInterleaved>
__device__ __forceinline__ uint4 pack(const Pairs &z) {
  if constexpr (kInterleaved)
    return make_uint4(bf16x2(low(z.a[0]), low(z.b[0])), bf16x2(high(z.a[0]), high(z.b[0])), bf16x2(low(z.a[1]), low(z.b[1])),
                      bf16x2(high(z.a[1]), high(z.b[1])));
  else
    return make_uint4(bf16x2(low(z.a[0]), high(z.a[0])), bf16x2(low(z.a[1]), high(z.a[1])), bf16x2(low(z.b[0]), high(z.b[0])),
                      bf16x2(low(z.b[1]), high(z.b[1])));
}
// Copies a lane's eight bf16 values of a head to its own place in shared memory, asynchronously:
// one copy, or two for halves.
template <bool kInterleaved>
__device__ __forceinline__ void copy_async(uint4 *to, const uint16_t *head, const Place &at) {
  const uint32_t dst = smem_u32(to);
  if constexpr (kInterleaved) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(head + at.a) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(head + at.a) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + 8), "l"(head + at.b) : "memory");
  }
}
template <bool kInterleaved>
__device__ __forceinline__ void store(uint16_t *head, const Place &at, const uint4 &v) {
  if constexpr (kInterleaved) {
    *reinterpret_cast<uint4 *>(head + at.a) = v;
  } else {
    *reinterpret_cast<uint2 *>(head + at.a) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2 *>(head + at.b) = make_uint2(v.z, v.w);
  }
}

// Four values of a lane's pairs from an array by dimension: halves, runs of four at a and b;
// interleaved, eight from a on.
template <bool kInterleaved>
__device__ __forceinline__ Pairs by_pairs(const Place &at, const float *v) {
  const float4 x = *reinterpret_cast<const float4 *>(v + at.a), y = *reinterpret_cast<const float4 *>(v + (kInterleaved ? at.a + 4 : at.b));
  Pairs p;
  if constexpr (kInterleaved) {
    p.a[0] = pack2(x.x, x.z);
    p.b[0] = pack2(x.y, x.w);
    p.a[1] = pack2(y.x, y.z);
    p.b[1] = pack2(y.y, y.w);
  } else {
    p.a[0] = pack2(x.x, x.y);
    p.a[1] = pack2(x.z, x.w);
    p.b[0] = pack2(y.x, y.y);
    p.b[1] = pack2(y.z, y.w);
  }
  return p;
}
// Deviations from the mean (kMean) and the mean of their squares.
template <int D, bool kMean>
__device__ __forceinline__ float spread(Pairs &x) {
  constexpr int kLanes = D / 8;
  if constexpr (kMean) {
    const uint64_t one = both(1.0f), t = fma2(fma2(x.a[0], one, x.a[1]), one, fma2(x.b[0], one, x.b[1]));
    const uint64_t minus = both(group_sum<kLanes>(low(t) + high(t)) * (-1.0f / D));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x.a[h] = fma2(x.a[h], one, minus);
      x.b[h] = fma2(x.b[h], one, minus);
    }
  }
  const uint64_t q = fma2(x.b[1], x.b[1], fma2(x.b[0], x.b[0], fma2(x.a[1], x.a[1], mul2(x.a[0], x.a[0]))));
  return group_sum<kLanes>(low(q) + high(q)) * (1.0f / D);
}

// 1 / sqrt of a normal number, to two units of the last place.
__device__ __forceinline__ float rsqrt_normal(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A head whose squares pass fp32's range: normed once more, scaled down by 2^80, beside which
// eps is nothing.  (A true infinity or NaN comes out as it would have.)  The whole warp calls.
struct Rescued {
  Pairs x;
  float inv;
};
template <int D, bool kInterleaved, bool kMean>
__device__ __noinline__ Rescued rescue(uint4 raw) {
  Rescued r;
  r.x = unpack<kInterleaved>(raw);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    r.x.a[h] = mul2(r.x.a[h], both(0x1p-80f));
    r.x.b[h] = mul2(r.x.b[h], both(0x1p-80f));
  }
  const float v = spread<D, kMean>(r.x);
  r.inv = v == 0.0f ? 0.0f : rsqrtf(v);   // equal elements whose sum passes the range: they deviate by 0
  return r;
}

// x to its normed values but for weights and biases and the factor `inv`.  The whole warp calls.
template <int D, bool kInterleaved, bool kMean>
__device__ __forceinline__ void normed(Pairs &x, const uint4 &raw, float eps, float &inv) {
  const float s = spread<D, kMean>(x);
  const bool past = !(s <= 3.402823466e38f);
  inv = rsqrt_normal(s + eps);
  if (__any_sync(0xffffffffu, past)) {
    const Rescued r = rescue<D, kInterleaved, kMean>(raw);
    if (past) {
      x = r.x;
      inv = r.inv;
    }
  }
}

// Cosines, sines and negated sines of a lane's four pairs, two in a word.
struct Turns {
  uint64_t c[2], s[2], m[2];
};
// Lanes of a warp with the same pairs, one in each head, work out a part of them each.
template <int D, bool kInterleaved>
__device__ __forceinline__ Turns turns_of(const idx_norm_rope_args &p, int64_t row, const Place &at) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x % 32 / kLanes;
  float2 mine[4 / kAtOnce];
#pragma unroll
  for (int j = 0; j < 4 / kAtOnce; ++j) {
    mine[j] = make_float2(1.0f, 0.0f);
    if (at.turns) {
      const int f = (kInterleaved ? at.a / 2 : at.a) + j * kAtOnce + sub;
      mine[j] = cos_sin(p.pos[p.axis[f] * p.pos_stride + row], p.inv_freq[f]);
    }
  }
  float c[4], s[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int from = k % kAtOnce * kLanes + lane;
    c[k] = __shfl_sync(0xffffffffu, mine[k / kAtOnce].x, from);
    s[k] = __shfl_sync(0xffffffffu, mine[k / kAtOnce].y, from);
  }
  Turns t;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    t.c[h] = pack2(c[2 * h], c[2 * h + 1]);
    t.s[h] = pack2(s[2 * h], s[2 * h + 1]);
    t.m[h] = pack2(-s[2 * h], -s[2 * h + 1]);
  }
  return t;
}
// A head's normed values, y, turned.
__device__ __forceinline__ Pairs turned(const Pairs &y, const Turns &t, const Place &at) {
  if (!at.turns) return y;
  Pairs z;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    z.a[h] = fma2(y.b[h], t.m[h], mul2(y.a[h], t.c[h]));
    z.b[h] = fma2(y.a[h], t.s[h], mul2(y.b[h], t.c[h]));
  }
  return z;
}

constexpr int ctas_per_sm(bool bias) { return bias ? 5 : 7; }   // 96 or 72 registers a thread

// A row's place in the cache for keys or values, at head h.
struct Spot {
  char *to;
  float *scale;
  bool live;
};
__device__ __forceinline__ Spot spot_of(const NormRopeArgs &a, bool values, bool f8, int64_t row, int h) {
  const uint32_t slot = static_cast<uint32_t>(a.p.slot[row]);   // negative slots are large ones
  const int64_t page = slot / kPage, tok = slot % kPage;
  Spot s;
  s.live = slot < static_cast<uint64_t>(a.c.P) * kPage;
  s.to = static_cast<char *>(values ? a.c.v : a.c.k) + (page * a.c.page_stride + tok * a.c.token_stride + h * a.c.head_stride) * (f8 ? 1 : 2);
  s.scale = f8 ? (values ? a.c.v_scale : a.c.k_scale) + (page * a.p.Hkv + h) * kPage + tok : nullptr;
  return s;
}

// Copies of batch `item` of a row, counted over all kinds (q's, then k's, then v's; none past the last).
template <int D, bool kInterleaved>
__device__ __forceinline__ void copy_item(const NormRopeArgs &a, int64_t row, int item, uint4 (&to)[kVectors][32]) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x % 32 / kLanes, slot = threadIdx.x % 32;
  const bool is_q = item < a.q_units, is_v = item >= a.q_units + a.k_units;
  if (is_v && (a.c.v == nullptr || item >= a.q_units + 2 * a.k_units)) return;
  const int u = is_q ? item : item - a.q_units - (is_v ? a.k_units : 0), first = u * a.heads;
  const int n = min((is_q ? a.p.Hq : a.p.Hkv) - first, a.heads) - sub;   // this lane's heads: 0, kAtOnce, .. below this
  const uint16_t *const src = static_cast<const uint16_t *>(is_q ? a.p.q : is_v ? a.p.v : a.p.k) +
                              row * (is_q ? a.p.q_stride : is_v ? a.p.v_stride : a.p.k_stride) + (first + sub) * D;
  const Place at = place_of<kInterleaved>(lane, a.p.rot);
#pragma unroll
  for (int k = 0; k < kVectors; ++k) {
    if (k * kAtOnce >= n) break;
    if (kInterleaved || !is_v) copy_async<kInterleaved>(&to[k][slot], src + k * kAtOnce * D, at);
    else copy_async<true>(&to[k][slot], src + k * kAtOnce * D, Place{8 * lane, 0, false});
  }
}

// Norm and rotation of a row's batches of one kind from `item` (over all kinds) on, whose copies to
// ring[stage] are on their way.  The first batch past them is on its way to the new ring[stage] then.
template <int D, bool kInterleaved, bool kBias, bool kKeys>
__device__ __forceinline__ void turn_items(const NormRopeArgs &a, int64_t row, int &item, int step, const Turns &turns, const Place &at,
                                           uint4 (*ring)[kVectors][32], int &stage) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kStep = kAtOnce * D;
  const idx_norm_rope_args &p = a.p;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x % 32 / kLanes, slot = threadIdx.x % 32;
  const int begin = kKeys ? a.q_units : 0, end = kKeys ? a.q_units + a.k_units : a.q_units;
  const int norm = kKeys ? p.k_norm : p.q_norm, heads = kKeys ? p.Hkv : p.Hq;
  if (item >= end) return;
  const float *const weight = kKeys ? p.k_weight : p.q_weight, *const bias = kKeys ? p.k_bias : p.q_bias;
  Pairs w, b;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w.a[h] = w.b[h] = both(1.0f);
    b.a[h] = b.b[h] = both(-0.0f);   // adds nothing to any value, a zero's sign included
  }
  if (weight != nullptr) w = by_pairs<kInterleaved>(at, weight);
  if (kBias && bias != nullptr) b = by_pairs<kInterleaved>(at, bias);
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3;
  uint16_t *const out = static_cast<uint16_t *>(kKeys ? p.k_out : p.q_out);
  uint16_t *const out0 = out + row * (kKeys ? p.k_out_stride : p.q_out_stride) + sub * D;
  Spot spot{};
  if (kKeys && p.slot != nullptr) spot = spot_of(a, false, f8, row, sub);
  // the next batch is on its way while one is worked on; a lane reads what it copied itself
#pragma unroll 1
  for (; item < end; item += step, stage ^= 1) {
    copy_item<D, kInterleaved>(a, row, item + step, ring[stage ^ 1]);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const int first = (item - begin) * a.heads, mine = min(heads - first, a.heads) - sub;
    uint16_t *const dst = out0 + first * D;
    char *const to = spot.to + first * a.c.head_stride * (f8 ? 1 : 2);
    const int64_t to_step = kAtOnce * a.c.head_stride * (f8 ? 1 : 2);
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
      if (k * kAtOnce >= mine + sub) break;   // the warp's lanes together
      const uint4 v = ring[stage][k][slot];   // past the last head: whatever is there, and not stored
      Pairs x = unpack<kInterleaved>(v);
      float inv = 1.0f;
      if (kBias && norm == IDX_NORM_LAYER) normed<D, kInterleaved, true>(x, v, p.eps, inv);
      else if (norm != IDX_NORM_NONE) normed<D, kInterleaved, false>(x, v, p.eps, inv);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x.a[h] = mul2(x.a[h], both(inv));
        x.b[h] = mul2(x.b[h], both(inv));
        if constexpr (kBias) {
          x.a[h] = fma2(x.a[h], w.a[h], b.a[h]);
          x.b[h] = fma2(x.b[h], w.b[h], b.b[h]);
        } else {
          x.a[h] = mul2(x.a[h], w.a[h]);
          x.b[h] = mul2(x.b[h], w.b[h]);
        }
      }
      const Pairs z = turned(x, turns, at);
      const uint4 packed = pack<kInterleaved>(z);
      const bool here = k * kAtOnce < mine;
      if ((!kKeys || out != nullptr) && here) store<kInterleaved>(dst + k * kStep, at, packed);
      if (!kKeys || spot.to == nullptr) continue;
      char *const head = to + k * to_step;
      if (!f8) {
        if (spot.live && here) store<kInterleaved>(reinterpret_cast<uint16_t *>(head), at, packed);
        continue;
      }
      // eight values in the order of their bytes
      const float e[8] = {low(z.a[0]), kInterleaved ? low(z.b[0]) : high(z.a[0]), kInterleaved ? high(z.a[0]) : low(z.a[1]),
                          kInterleaved ? high(z.b[0]) : high(z.a[1]), kInterleaved ? low(z.a[1]) : low(z.b[0]),
                          kInterleaved ? low(z.b[1]) : high(z.b[0]), kInterleaved ? high(z.a[1]) : low(z.b[1]), high(z.b[1])};
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(e[j]));
      uint32_t lo, hi;
      const float sc = quantize_f32(e, group_max<kLanes>(m), lo, hi);
      if (spot.live && here) {
        if (kInterleaved) {
          *reinterpret_cast<uint2 *>(head + at.a) = make_uint2(lo, hi);
        } else {
          *reinterpret_cast<uint32_t *>(head + at.a) = lo;
          *reinterpret_cast<uint32_t *>(head + at.b) = hi;
        }
        if (lane == 0) spot.scale[(first + k * kAtOnce) * kPage] = sc;
      }
    }
  }
}

// kBias: a LayerNorm is among the norms.
template <int D, bool kInterleaved, bool kBias>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kBias)) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  __shared__ uint4 rings[kWarps][2][kVectors][32];
  const idx_norm_rope_args &p = a.p;
  const int tid = threadIdx.x, lane = tid % kLanes, sub = tid % 32 / kLanes, slot = tid % 32;
  const uint32_t index = blockIdx.x * kWarps + tid / 32;   // R * parts is below 2^31
  const int64_t row = index / static_cast<uint32_t>(a.parts);
  const int step = a.parts;
  int item = static_cast<int>(index % static_cast<uint32_t>(a.parts)), stage = 0;
  uint4(*const ring)[kVectors][32] = rings[tid / 32];
  grid_dependency_trigger();
  grid_dependency_wait();
  if (row >= p.R || (p.rows != nullptr && row >= *p.rows)) return;

  // the warp's first copies, before the angles
  copy_item<D, kInterleaved>(a, row, item, ring[0]);
  asm volatile("cp.async.commit_group;" ::: "memory");
  const Place at = place_of<kInterleaved>(lane, p.rot);
  if (item < a.q_units + a.k_units) {
    const Turns turns = turns_of<D, kInterleaved>(p, row, at);
    turn_items<D, kInterleaved, kBias, false>(a, row, item, step, turns, at, ring, stage);
    turn_items<D, kInterleaved, kBias, true>(a, row, item, step, turns, at, ring, stage);
  }
  const int end = a.q_units + 2 * a.k_units;
  if (a.c.v == nullptr || item >= end) return;
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3;
  const Spot spot = spot_of(a, true, f8, row, sub);
  const int64_t to_step = kAtOnce * a.c.head_stride * (f8 ? 1 : 2);
#pragma unroll 1
  for (; item < end; item += step, stage ^= 1) {
    copy_item<D, kInterleaved>(a, row, item + step, ring[stage ^ 1]);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const int first = (item - a.q_units - a.k_units) * a.heads, mine = min(p.Hkv - first, a.heads) - sub;
    char *const to = spot.to + first * a.c.head_stride * (f8 ? 1 : 2);
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
      if (k * kAtOnce >= mine + sub) break;   // the warp's lanes together
      const bool here = spot.live && k * kAtOnce < mine;
      char *const head = to + k * to_step;
      const uint4 v = ring[stage][k][slot];
      if (f8) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t lo, hi;
        const float sc = quantize(w, vector_amax<kLanes>(w), lo, hi);
        if (here) {
          *reinterpret_cast<uint2 *>(head + 8 * lane) = make_uint2(lo, hi);
          if (lane == 0) spot.scale[(first + k * kAtOnce) * kPage] = sc;
        }
      } else if (here) {
        *reinterpret_cast<uint4 *>(head + 16 * lane) = v;
      }
    }
  }
}

template <int D, bool kInterleaved, bool kBias>
cudaError_t launch(NormRopeArgs a, int num_sms, cudaStream_t stream) {
  constexpr int kAtOnce = 32 / (D / 8);
  const int kinds = a.c.v != nullptr ? 2 : 1;
  // Batches as large as leaves each of the warps that run at a time one, and a row to a warp where there
  // are as many rows.
  const int64_t warps = static_cast<int64_t>(num_sms) * ctas_per_sm(kBias) * kWarps;
  for (int per = 1;; per *= 2) {
    a.heads = per * kAtOnce;
    a.q_units = (a.p.Hq + a.heads - 1) / a.heads;
    a.k_units = (a.p.Hkv + a.heads - 1) / a.heads;
    a.parts = a.q_units + a.k_units * kinds;
    if (per == kVectors || 2 * a.p.R * a.parts <= warps) break;
  }
  a.parts = static_cast<int>(std::min<int64_t>(a.parts, (warps + a.p.R - 1) / a.p.R));
  const int64_t grid = (a.p.R * a.parts + kWarps - 1) / kWarps;
  return launch_early(norm_rope_kernel<D, kInterleaved, kBias>, static_cast<unsigned>(grid), kThreads, 0, 1, stream, a);
}

template <int D>
cudaError_t launch(const NormRopeArgs &a, int num_sms, cudaStream_t stream) {
  const bool il = a.p.interleaved != 0, ln = a.p.q_norm == IDX_NORM_LAYER || a.p.k_norm == IDX_NORM_LAYER;
  if (ln) return il ? launch<D, true, true>(a, num_sms, stream) : launch<D, false, true>(a, num_sms, stream);
  return il ? launch<D, true, false>(a, num_sms, stream) : launch<D, false, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, int num_sms, cudaStream_t stream) {
  return a.p.D == 64 ? launch<64>(a, num_sms, stream) : a.p.D == 128 ? launch<128>(a, num_sms, stream) : launch<256>(a, num_sms, stream);
}

}  // namespace idx
