// Norms of queries and keys for each head, their rotation, and keys and values into the
// paged cache, in one pass over a projection's output.
//
// A vector of D values (one head of a row) is a group of D / 8 lanes with eight values each,
// four pairs that turn together, so that the rotation stays within a lane: two runs of four
// for halves, one of eight for interleaved pairs.  It is read once and written once.  A CTA
// takes a group of rows, works their angles out once into shared memory, and its warps walk
// over units of a few heads of a row of one kind (q, k or v).  The rotation is linear in the
// normed head, y = inv * (x - mean) * w + b, so weight, bias, cosine and sine fold into a
// unit's factors: for a pair (a, b)
//     z_a = inv * ((a - mean) w_a c - (b - mean) w_b s) + (b_a c - b_b s),
// and z_b alike.
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
constexpr int kVectors = 4;     // loads of a lane in flight
constexpr int kMostRows = 8;    // of a CTA's group
constexpr int kCtasPerSm = 3;

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
// A lane's eight bf16 values of a head: one load for interleaved pairs, two for halves.
template <bool kInterleaved>
__device__ __forceinline__ uint4 load(const uint16_t *head, const Place &at) {
  if constexpr (kInterleaved) return __ldcs(reinterpret_cast<const uint4 *>(head + at.a));
  const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(head + at.a)), b = __ldcs(reinterpret_cast<const uint2 *>(head + at.b));
  return make_uint4(a.x, a.y, b.x, b.y);
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

// A unit's factors for a lane: z_a = inv (x_a aa + x_b ab) + ca, z_b = inv (x_b bb + x_a ba) + cb.
struct Factors {
  uint64_t aa[2], ab[2], bb[2], ba[2], ca[2], cb[2];
};
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
// cs: the row's (cos, sin) per frequency; w, b: the head's weights and biases in shared memory.
template <bool kInterleaved, bool kBias>
__device__ __forceinline__ void make_factors(const Place &at, const float2 *cs, const float *w, const float *b, Factors &f) {
  float4 t[2] = {make_float4(1.0f, 0.0f, 1.0f, 0.0f), make_float4(1.0f, 0.0f, 1.0f, 0.0f)};
  if (at.turns) {
    const float4 *const from = reinterpret_cast<const float4 *>(cs + (kInterleaved ? at.a / 2 : at.a));   // four frequencies
    t[0] = from[0];
    t[1] = from[1];
  }
  const Pairs v = by_pairs<kInterleaved>(at, w);
  Pairs u{};
  if constexpr (kBias) u = by_pairs<kInterleaved>(at, b);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t c = pack2(t[h].x, t[h].z), s = pack2(t[h].y, t[h].w), m = pack2(-t[h].y, -t[h].w);
    f.aa[h] = mul2(v.a[h], c);
    f.ab[h] = mul2(v.b[h], m);
    f.bb[h] = mul2(v.b[h], c);
    f.ba[h] = mul2(v.a[h], s);
    if (!at.turns) f.ab[h] = f.ba[h] = both(-0.0f);   // times 0: adds nothing, a zero's sign included
    if constexpr (kBias) {
      f.ca[h] = at.turns ? fma2(u.b[h], m, mul2(u.a[h], c)) : u.a[h];
      f.cb[h] = at.turns ? fma2(u.a[h], s, mul2(u.b[h], c)) : u.b[h];
    }
  }
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

// x of kAtATime heads to their normed values but for weights and biases.  The whole warp calls.
template <int D, bool kMean, int kAtATime>
__device__ __forceinline__ void normed(Pairs (&x)[kAtATime], const uint4 (&raw)[kAtATime], bool interleaved, float eps, float (&inv)[kAtATime]) {
  float s[kAtATime];
  bool again = false;
#pragma unroll
  for (int k = 0; k < kAtATime; ++k) {
    s[k] = spread<D, kMean>(x[k]);
    again = again || !(s[k] <= 3.402823466e38f);
    inv[k] = rsqrtf(s[k] + eps);
  }
  // Squares past fp32's range: once more with the head scaled down by 2^80, beside which eps is
  // nothing.  (A true infinity or NaN comes out the same way the second time.)
  if (__any_sync(0xffffffffu, again)) {
#pragma unroll
    for (int k = 0; k < kAtATime; ++k) {
      Pairs y = interleaved ? unpack<true>(raw[k]) : unpack<false>(raw[k]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        y.a[h] = mul2(y.a[h], both(0x1p-80f));
        y.b[h] = mul2(y.b[h], both(0x1p-80f));
      }
      const float t = spread<D, kMean>(y);
      if (!(s[k] <= 3.402823466e38f)) {
        x[k] = y;
        inv[k] = rsqrtf(t);
      }
    }
  }
}

// A head's values turned by their factors.
template <bool kBias>
__device__ __forceinline__ Pairs turned(const Pairs &x, const Factors &f, float inv, bool crosses) {
  Pairs z;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // where nothing turns, the other's factor is 0: an infinite other must not make it NaN
    const uint64_t oa = crosses ? x.b[h] : 0, ob = crosses ? x.a[h] : 0;
    const uint64_t ta = fma2(x.a[h], f.aa[h], mul2(oa, f.ab[h])), tb = fma2(x.b[h], f.bb[h], mul2(ob, f.ba[h]));
    if constexpr (kBias) {
      z.a[h] = fma2(both(inv), ta, f.ca[h]);
      z.b[h] = fma2(both(inv), tb, f.cb[h]);
    } else {
      z.a[h] = mul2(both(inv), ta);
      z.b[h] = mul2(both(inv), tb);
    }
  }
  return z;
}

// kBias: a LayerNorm is among the norms.
template <int D, bool kInterleaved, bool kBias>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  constexpr int kPair = kBias ? 1 : 2;   // heads normed at a time, so that one's sums run beside the other's
  __shared__ __align__(16) float2 cs[kMostRows][D / 2];
  __shared__ __align__(16) float weights[2][D], biases[kBias ? 2 : 1][kBias ? D : 4];   // of q and of k
  const idx_norm_rope_args &p = a.p;
  const int tid = threadIdx.x, lane = tid % kLanes, sub = tid % 32 / kLanes, warp = tid / 32;
  const int64_t group = blockIdx.x / a.splits;
  const int part = static_cast<int>(blockIdx.x % a.splits);
  const int64_t row0 = group * a.group_rows;
  const int64_t limit = p.rows != nullptr ? min(p.R, static_cast<int64_t>(*p.rows)) : p.R;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.group_rows), limit - row0));
  if (rows <= 0) return;

  const int pairs = p.rot >> 1;
  for (int i = tid; i < rows * pairs; i += kThreads) {
    const int r = i / pairs, k = i % pairs;
    cs[r][k] = cos_sin(p.pos[p.axis[k] * p.pos_stride + row0 + r], p.inv_freq[k]);
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

  const Place at = place_of<kInterleaved>(lane, p.rot);
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3, crosses = p.rot == D || at.turns;
  constexpr int kStep = kAtOnce * D;   // elements from one of a lane's heads to the next
  int r = 0, u = part * kWarps + warp;
  for (; u >= a.units; u -= a.units) ++r;
  while (r < rows) {
    const int64_t row = row0 + r;
    // the unit's kind and heads: this lane's are h, h + kAtOnce, ..., `mine` of them
    const int kind = u < a.q_units ? 0 : u < a.q_units + a.k_units ? 1 : 2;
    const int first = (u - (kind == 0 ? 0 : kind == 1 ? a.q_units : a.q_units + a.k_units)) * a.heads, h = first + sub;
    const int heads = min(a.heads, (kind == 0 ? p.Hq : p.Hkv) - first), mine = (heads - sub + kAtOnce - 1) / kAtOnce;
    const uint16_t *const src = static_cast<const uint16_t *>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                                row * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride) + h * D;
    uint4 raw[kVectors];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
      raw[k] = make_uint4(0u, 0u, 0u, 0u);
      if (k < mine) raw[k] = kind == 2 ? __ldcs(reinterpret_cast<const uint4 *>(src + k * kStep + 8 * lane)) : load<kInterleaved>(src + k * kStep, at);
    }

    // the row's place in the cache, at head h
    char *to = nullptr;
    float *scale = nullptr;
    bool live = false;
    if (kind != 0 && p.slot != nullptr) {
      const uint32_t slot = static_cast<uint32_t>(p.slot[row]);   // negative slots are large ones
      live = slot < static_cast<uint64_t>(a.c.P) * kPage;
      const int64_t page = slot / kPage, tok = slot % kPage;
      to = static_cast<char *>(kind == 1 ? a.c.k : a.c.v) +
           (page * a.c.page_stride + tok * a.c.token_stride + h * a.c.head_stride) * (f8 ? 1 : 2);
      scale = f8 ? (kind == 1 ? a.c.k_scale : a.c.v_scale) + (page * p.Hkv + h) * kPage + tok : nullptr;
    }
    const int64_t to_step = kAtOnce * a.c.head_stride * (f8 ? 1 : 2);

    if (kind == 2) {
#pragma unroll
      for (int k = 0; k < kVectors; ++k) {
        if (k * kAtOnce >= heads) break;   // the warp's lanes together
        if (f8) {
          const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
          uint32_t lo, hi;
          const float sc = quantize(w, vector_amax<kLanes>(w), lo, hi);
          if (live && k < mine) {
            *reinterpret_cast<uint2 *>(to + k * to_step + 8 * lane) = make_uint2(lo, hi);
            if (lane == 0) scale[k * kAtOnce * kPage] = sc;
          }
        } else if (live && k < mine) {
          *reinterpret_cast<uint4 *>(to + k * to_step + 16 * lane) = raw[k];
        }
      }
    } else {
      uint16_t *dst = static_cast<uint16_t *>(kind == 0 ? p.q_out : p.k_out);
      const bool out = dst != nullptr;
      if (out) dst += row * (kind == 0 ? p.q_out_stride : p.k_out_stride) + h * D;
      Factors f;
      make_factors<kInterleaved, kBias>(at, cs[r], weights[kind], kBias ? biases[kind] : nullptr, f);
      const int norm = kind == 0 ? p.q_norm : p.k_norm;
#pragma unroll
      for (int k0 = 0; k0 < kVectors; k0 += kPair) {
        if (k0 * kAtOnce >= heads) break;   // the warp's lanes together
        Pairs x[kPair];
        uint4 v[kPair];
        float inv[kPair];
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          v[k] = raw[k0 + k];
          x[k] = unpack<kInterleaved>(v[k]);
          inv[k] = 1.0f;
        }
        if (kBias && norm == IDX_NORM_LAYER) normed<D, true>(x, v, kInterleaved, p.eps, inv);
        else if (norm != IDX_NORM_NONE) normed<D, false>(x, v, kInterleaved, p.eps, inv);
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          const Pairs z = turned<kBias>(x[k], f, inv[k], crosses);
          const uint4 packed = pack<kInterleaved>(z);
          const bool here = k0 + k < mine;
          if (out && here) store<kInterleaved>(dst + (k0 + k) * kStep, at, packed);
          if (to == nullptr) continue;
          char *const head = to + (k0 + k) * to_step;
          if (!f8) {
            if (live && here) store<kInterleaved>(reinterpret_cast<uint16_t *>(head), at, packed);
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
          if (live && here) {
            if (kInterleaved) {
              *reinterpret_cast<uint2 *>(head + at.a) = make_uint2(lo, hi);
            } else {
              *reinterpret_cast<uint32_t *>(head + at.a) = lo;
              *reinterpret_cast<uint32_t *>(head + at.b) = hi;
            }
            if (lane == 0) scale[(k0 + k) * kAtOnce * kPage] = sc;
          }
        }
      }
    }
    for (u += a.splits * kWarps; u >= a.units; u -= a.units) ++r;
  }
}

template <int D, bool kInterleaved, bool kBias>
cudaError_t launch(NormRopeArgs a, int num_sms, cudaStream_t stream) {
  constexpr int kAtOnce = 32 / (D / 8);
  const int kinds = a.c.v != nullptr ? 2 : 1;
  // Units of kVectors loads a lane and groups of kMostRows rows where that leaves every SM its
  // CTAs; else single loads, single rows and as many CTAs to a row as it has warps of work.
  const int64_t vectors = a.p.R * (a.p.Hq + static_cast<int64_t>(a.p.Hkv) * kinds);
  const int64_t full = static_cast<int64_t>(num_sms) * kCtasPerSm * kWarps * kAtOnce;   // vectors that the GPU holds
  int per = 1;
  while (per < kVectors && vectors >= 2 * per * full) per *= 2;
  a.heads = per * kAtOnce;
  a.q_units = (a.p.Hq + a.heads - 1) / a.heads;
  a.k_units = (a.p.Hkv + a.heads - 1) / a.heads;
  a.units = a.q_units + a.k_units * kinds;
  a.group_rows = 1;
  while (a.group_rows < kMostRows && a.p.R >= 2 * a.group_rows * static_cast<int64_t>(num_sms) * kCtasPerSm) a.group_rows *= 2;
  a.splits = 1;
  if (a.group_rows == 1) a.splits = (a.units + kWarps - 1) / kWarps;
  const int64_t grid = (a.p.R + a.group_rows - 1) / a.group_rows * a.splits;
  norm_rope_kernel<D, kInterleaved, kBias><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
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
