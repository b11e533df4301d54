// Norms of queries and keys for each head, their rotation, and keys and values into the
// paged cache, in one pass over a projection's output.
//
// A vector of D values (one head of a row) is a group of D / 8 lanes with eight values each,
// four pairs that turn together, so that the rotation stays within a lane: two runs of four
// for halves, one of eight for interleaved pairs.  It is read once and written once.  A CTA
// takes a group of rows, works their angles out once into shared memory, and its warps take
// batches of a few heads of one row, first of q, then of k, then of v, each in a loop of its
// own that keeps the head's weights in registers (one walk over all kinds, with its branches and
// reloads, took 152 us for the prompts below; loops by kind with the next batch's copies on
// their way 114).  A warp takes every `step`-th batch: runs of consecutive batches left warps with
// uneven ends and were slower.
//
// What bounds it: 16,209 prompt rows of 64 + 2 x 8 heads of 128 into an E4M3 cache take 113.6 us,
// 5.6 TB/s or 82% of the measured copy bandwidth, with 60% of the issue slots busy, so everything is
// done for two values at a time.  8,855 rows of 16 + 2 x 16 heads turned by three axes, bf16: 42.9 us, 75%.
// A few rows: 3.4 us in a graph, which is launch, one read and one write.
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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVectors = 4;     // heads of a lane in a batch
constexpr int kMostRows = 8;    // of a CTA's group

// inv_freq / (2 pi) in units of 2^-64 turn, modulo one turn: the 24-bit significand times
// 2^64 / (2 pi), shifted by the exponent.
__device__ __forceinline__ uint64_t turns_per_position(float inv_freq) {
  constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;   // 2^64 / (2 pi)
  const uint32_t u = __float_as_uint(inv_freq);
  const uint32_t ex = (u >> 23) & 0xFFu;
  const uint64_t m = (u & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int down = 150 - static_cast<int>(ex ? ex : 1u);   // the value is m * 2^-down
  uint64_t f;
  if (down <= 0) f = -down < 64 ? lo << -down : 0ull;
  else if (down < 64) f = lo >> down | hi << (64 - down);
  else f = down < 128 ? hi >> (down - 64) : 0ull;
  return u >> 31 ? 0ull - f : f;
}

__device__ __forceinline__ float2 cos_sin(int32_t pos, float inv_freq) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns_per_position(inv_freq);
  // the nearest quarter turn, and what is left of it, within an eighth: 32 of the 64 bits,
  // rounded to fp32 at that smaller size
  const uint32_t turn = static_cast<uint32_t>(phase >> 32), quarter = (turn + 0x20000000u) >> 30;
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
  r.inv = rsqrtf(spread<D, kMean>(r.x));
  return r;
}

// x of kAtATime heads to their normed values but for weights and biases.  The whole warp calls.
template <int D, bool kInterleaved, bool kMean, int kAtATime>
__device__ __forceinline__ void normed(Pairs (&x)[kAtATime], const uint4 (&raw)[kAtATime], float eps, float (&inv)[kAtATime]) {
  float s[kAtATime];
  bool past = false;
#pragma unroll
  for (int k = 0; k < kAtATime; ++k) {
    s[k] = spread<D, kMean>(x[k]);
    past = past || !(s[k] <= 3.402823466e38f);
    inv[k] = rsqrt_normal(s[k] + eps);
  }
  if (__any_sync(0xffffffffu, past)) {
#pragma unroll
    for (int k = 0; k < kAtATime; ++k) {
      const Rescued r = rescue<D, kInterleaved, kMean>(raw[k]);
      if (!(s[k] <= 3.402823466e38f)) {
        x[k] = r.x;
        inv[k] = r.inv;
      }
    }
  }
}

// Cosines, sines and negated sines of a row's frequencies, each in a run.
template <int D>
struct Turns {
  float c[D / 2], s[D / 2], m[D / 2];
};
// A head's normed values, y, turned, times inv.
template <int D, bool kInterleaved>
__device__ __forceinline__ Pairs turned(const Pairs &y, const Turns<D> &t, const Place &at) {
  if (!at.turns) return y;
  const int f = kInterleaved ? at.a / 2 : at.a;   // four frequencies
  const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(t.c + f), s = *reinterpret_cast<const ulonglong2 *>(t.s + f),
                   m = *reinterpret_cast<const ulonglong2 *>(t.m + f);
  Pairs z;
  z.a[0] = fma2(y.b[0], m.x, mul2(y.a[0], c.x));
  z.a[1] = fma2(y.b[1], m.y, mul2(y.a[1], c.y));
  z.b[0] = fma2(y.a[0], s.x, mul2(y.b[0], c.x));
  z.b[1] = fma2(y.a[1], s.y, mul2(y.b[1], c.y));
  return z;
}

constexpr int ctas_per_sm(bool bias) { return bias ? 2 : 3; }   // 128 or 80 registers a thread

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

// A warp's batches of one kind (0 q, 1 k, 2 v) in a group of rows: item i is batch i % units of
// row i / units, a step from one to the next; and the copies that run one batch ahead.
template <int D, bool kInterleaved, int kKind>
struct Walk {
  static constexpr int kAtOnce = 32 / (D / 8);
  const NormRopeArgs &a;
  const int units, heads, step;
  const uint16_t *const in;   // the group's first row, this lane's first head
  const int64_t stride;
  const Place at;
  int r, u, r_next, u_next;

  __device__ __forceinline__ Walk(const NormRopeArgs &args, int64_t row0, int item, int step_)
      : a(args), units(kKind == 0 ? args.q_units : args.k_units), heads(kKind == 0 ? args.p.Hq : args.p.Hkv), step(step_),
        in(static_cast<const uint16_t *>(kKind == 0 ? args.p.q : kKind == 1 ? args.p.k : args.p.v) +
           row0 * (kKind == 0 ? args.p.q_stride : kKind == 1 ? args.p.k_stride : args.p.v_stride) + sub() * D),
        stride(kKind == 0 ? args.p.q_stride : kKind == 1 ? args.p.k_stride : args.p.v_stride),
        at(kKind == 2 ? Place{8 * lane(), 0, false} : place_of<kInterleaved>(lane(), args.p.rot)) {
    r = r_next = item / units;
    u = u_next = item % units;
  }
  static __device__ __forceinline__ int lane() { return threadIdx.x % (D / 8); }
  static __device__ __forceinline__ int sub() { return threadIdx.x % 32 / (D / 8); }
  __device__ __forceinline__ int first() const { return u * a.heads; }
  // This lane's heads of the batch: 0, kAtOnce, .. below this.
  __device__ __forceinline__ int mine(int batch) const { return min(heads - batch * a.heads - sub(), a.heads - sub()); }
  __device__ __forceinline__ void copy_next(uint4 (&to)[kVectors][32]) {
    const int n = mine(u_next);
    const uint16_t *const src = in + r_next * stride + u_next * a.heads * D;
#pragma unroll
    for (int k = 0; k < kVectors; ++k)
      if (k * kAtOnce < n) copy_async<kInterleaved || kKind == 2>(&to[k][threadIdx.x % 32], src + k * kAtOnce * D, at);
    for (u_next += step; u_next >= units; u_next -= units) ++r_next;
  }
  __device__ __forceinline__ void next() {
    for (u += step; u >= units; u -= units) ++r;
  }
};

// Norm and rotation of a kind's items from `item` on.  Returns the first item past them.
// copied: the first batch's copies are on their way.
template <int D, bool kInterleaved, bool kBias, bool kKeys>
__device__ __forceinline__ int turn_items(const NormRopeArgs &a, int item, int step, int rows, int64_t row0, const Turns<D> *turns,
                                          const float *weight, const float *bias, uint4 (*ring)[kVectors][32], bool copied) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kStep = kAtOnce * D;
  constexpr int kPair = kBias ? 1 : 2;   // heads normed at a time, so that one's sums run beside the other's
  const idx_norm_rope_args &p = a.p;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x % 32 / kLanes, slot = threadIdx.x % 32;
  const int items = rows * (kKeys ? a.k_units : a.q_units), norm = kKeys ? p.k_norm : p.q_norm;
  if (item >= items) return item - items;
  Walk<D, kInterleaved, kKeys ? 1 : 0> walk(a, row0, item, step);
  const Place &at = walk.at;
  const Pairs w = by_pairs<kInterleaved>(at, weight);
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3;
  uint16_t *const out = static_cast<uint16_t *>(kKeys ? p.k_out : p.q_out);
  uint16_t *const out0 = out + row0 * (kKeys ? p.k_out_stride : p.q_out_stride) + sub * D;
  // the next batch is on its way while one is worked on; a lane reads what it copied itself
  int stage = 0;
  if (copied) {
    for (walk.u_next += step; walk.u_next >= walk.units; walk.u_next -= walk.units) ++walk.r_next;
  } else {
    walk.copy_next(ring[0]);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
#pragma unroll 1
  for (; item < items; item += step, stage ^= 1, walk.next()) {
    if (item + step < items) walk.copy_next(ring[stage ^ 1]);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const int r = walk.r, first = walk.first(), mine = walk.mine(walk.u);
    uint16_t *const dst = out0 + r * (kKeys ? p.k_out_stride : p.q_out_stride) + first * D;
    Spot spot{};
    if (kKeys && p.slot != nullptr) spot = spot_of(a, false, f8, row0 + r, first + sub);
    const int64_t to_step = kAtOnce * a.c.head_stride * (f8 ? 1 : 2);
#pragma unroll
    for (int k0 = 0; k0 < kVectors; k0 += kPair) {
      if (k0 * kAtOnce >= mine + sub) break;   // the warp's lanes together
      Pairs x[kPair];
      uint4 v[kPair];
      float inv[kPair];
#pragma unroll
      for (int k = 0; k < kPair; ++k) {
        v[k] = ring[stage][k0 + k][slot];   // past the last head: whatever is there, and not stored
        x[k] = unpack<kInterleaved>(v[k]);
        inv[k] = 1.0f;
      }
      if (kBias && norm == IDX_NORM_LAYER) normed<D, kInterleaved, true>(x, v, p.eps, inv);
      else if (norm != IDX_NORM_NONE) normed<D, kInterleaved, false>(x, v, p.eps, inv);
#pragma unroll
      for (int k = 0; k < kPair; ++k) {
        Pairs y;
        if constexpr (kBias) {
          const Pairs b = by_pairs<kInterleaved>(at, bias);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            y.a[h] = fma2(mul2(x[k].a[h], both(inv[k])), w.a[h], b.a[h]);
            y.b[h] = fma2(mul2(x[k].b[h], both(inv[k])), w.b[h], b.b[h]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            y.a[h] = mul2(mul2(x[k].a[h], both(inv[k])), w.a[h]);
            y.b[h] = mul2(mul2(x[k].b[h], both(inv[k])), w.b[h]);
          }
        }
        const Pairs z = turned<D, kInterleaved>(y, turns[r], at);
        const uint4 packed = pack<kInterleaved>(z);
        const bool here = (k0 + k) * kAtOnce < mine;
        if ((!kKeys || out != nullptr) && here) store<kInterleaved>(dst + (k0 + k) * kStep, at, packed);
        if (!kKeys || spot.to == nullptr) continue;
        char *const head = spot.to + (k0 + k) * to_step;
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
          if (lane == 0) spot.scale[(k0 + k) * kAtOnce * kPage] = sc;
        }
      }
    }
  }
  return item - items;
}

// kBias: a LayerNorm is among the norms.
template <int D, bool kInterleaved, bool kBias>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kBias)) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  __shared__ __align__(16) Turns<D> turns[kMostRows];
  __shared__ uint4 rings[kWarps][2][kVectors][32];
  __shared__ __align__(16) float weights[2][D], biases[kBias ? 2 : 1][kBias ? D : 4];   // of q and of k
  const idx_norm_rope_args &p = a.p;
  const int tid = threadIdx.x;
  grid_dependency_trigger();
  grid_dependency_wait();
  const int64_t group = blockIdx.x / a.splits;
  const int part = static_cast<int>(blockIdx.x % a.splits);
  const int64_t row0 = group * a.group_rows;
  const int64_t limit = p.rows != nullptr ? min(p.R, static_cast<int64_t>(*p.rows)) : p.R;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.group_rows), limit - row0));
  if (rows <= 0) return;

  // the warp's first copies, before the angles
  const int step = a.splits * kWarps;
  int item = part * kWarps + tid / 32;
  uint4(*const ring)[kVectors][32] = rings[tid / 32];
  const int kind = item < rows * a.q_units ? 0 : item < rows * (a.q_units + a.k_units) ? 1 : 2;
  if (kind == 0) Walk<D, kInterleaved, 0>(a, row0, item, step).copy_next(ring[0]);
  if (kind == 1) Walk<D, kInterleaved, 1>(a, row0, item - rows * a.q_units, step).copy_next(ring[0]);
  asm volatile("cp.async.commit_group;" ::: "memory");

  const int pairs = p.rot >> 1;
  for (int i = tid; i < rows * pairs; i += kThreads) {
    const int r = i / pairs, k = i % pairs;
    const float2 t = cos_sin(p.pos[p.axis[k] * p.pos_stride + row0 + r], p.inv_freq[k]);
    turns[r].c[k] = t.x;
    turns[r].s[k] = t.y;
    turns[r].m[k] = -t.y;
  }
  for (int i = tid; i < D; i += kThreads) {
    weights[0][i] = p.q_weight != nullptr ? p.q_weight[i] : 1.0f;
    weights[1][i] = p.k_weight != nullptr ? p.k_weight[i] : 1.0f;
    if constexpr (kBias) {   // -0 adds nothing to any value, a zero's sign included
      biases[0][i] = p.q_bias != nullptr ? p.q_bias[i] : -0.0f;
      biases[1][i] = p.k_bias != nullptr ? p.k_bias[i] : -0.0f;
    }
  }
  __syncthreads();

  item = turn_items<D, kInterleaved, kBias, false>(a, item, step, rows, row0, turns, weights[0], biases[0], ring, kind == 0);
  item = turn_items<D, kInterleaved, kBias, true>(a, item, step, rows, row0, turns, weights[1], biases[kBias ? 1 : 0], ring, kind == 1);
  if (a.c.v == nullptr || item >= rows * a.k_units) return;
  Walk<D, kInterleaved, 2> walk(a, row0, item, step);
  const int lane = tid % kLanes, sub = tid % 32 / kLanes, slot = tid % 32;
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3;
  const int64_t to_step = kAtOnce * a.c.head_stride * (f8 ? 1 : 2);
  int stage = 0;
  walk.copy_next(ring[0]);
  asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 1
  for (; item < rows * a.k_units; item += step, stage ^= 1, walk.next()) {
    if (item + step < rows * a.k_units) walk.copy_next(ring[stage ^ 1]);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int first = walk.first(), mine = walk.mine(walk.u);
    const Spot spot = spot_of(a, true, f8, row0 + walk.r, first + sub);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
      if (k * kAtOnce >= mine + sub) break;   // the warp's lanes together
      const bool here = spot.live && k * kAtOnce < mine;
      char *const head = spot.to + k * to_step;
      const uint4 v = ring[stage][k][slot];
      if (f8) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t lo, hi;
        const float sc = quantize(w, vector_amax<kLanes>(w), lo, hi);
        if (here) {
          *reinterpret_cast<uint2 *>(head + 8 * lane) = make_uint2(lo, hi);
          if (lane == 0) spot.scale[k * kAtOnce * kPage] = sc;
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
  // Groups of kMostRows rows where that leaves every SM its CTAs, else of fewer; below that as
  // many CTAs to a row as run at a time, and batches as large as leaves each of their warps one.
  const int64_t ctas = static_cast<int64_t>(num_sms) * ctas_per_sm(kBias);
  a.group_rows = 1;
  while (a.group_rows < kMostRows && a.p.R >= 2 * a.group_rows * ctas) a.group_rows *= 2;
  const int most = static_cast<int>(std::max<int64_t>(1, ctas / a.p.R));
  int per = 1;
  for (;; per *= 2) {
    a.heads = per * kAtOnce;
    a.q_units = (a.p.Hq + a.heads - 1) / a.heads;
    a.k_units = (a.p.Hkv + a.heads - 1) / a.heads;
    a.splits = (a.q_units + a.k_units * kinds + kWarps - 1) / kWarps;
    if (per == kVectors || (a.group_rows == 1 && a.splits <= most)) break;
  }
  a.splits = a.group_rows > 1 ? 1 : std::min(a.splits, most);
  const int64_t grid = (a.p.R + a.group_rows - 1) / a.group_rows * a.splits;
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
