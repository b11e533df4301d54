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
// cs: the row's (cos, sin) per frequency; w, b: the head's weights and biases in shared memory.
template <bool kInterleaved, bool kBias>
__device__ __forceinline__ void make_factors(const Place &at, const float2 *cs, const float *w, const float *b, Factors &f) {
  constexpr int kStep = kInterleaved ? 2 : 1;
  const int first = kInterleaved ? at.a / 2 : at.a;   // of the lane's frequencies
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 t[2] = {make_float2(1.0f, 0.0f), make_float2(1.0f, 0.0f)};
    if (at.turns) {
      t[0] = cs[first + 2 * h];
      t[1] = cs[first + 2 * h + 1];
    }
    const uint64_t c = pack2(t[0].x, t[1].x), s = pack2(t[0].y, t[1].y), m = pack2(-t[0].y, -t[1].y);
    const uint64_t wa = pack2(w[at.a + kStep * 2 * h], w[at.a + kStep * (2 * h + 1)]);
    const uint64_t wb = pack2(w[at.b + kStep * 2 * h], w[at.b + kStep * (2 * h + 1)]);
    f.aa[h] = mul2(wa, c);
    f.ab[h] = mul2(wb, m);
    f.bb[h] = mul2(wb, c);
    f.ba[h] = mul2(wa, s);
    if (!at.turns) f.ab[h] = f.ba[h] = both(-0.0f);   // times 0: adds nothing, a zero's sign included
    if constexpr (kBias) {
      const uint64_t va = pack2(b[at.a + kStep * 2 * h], b[at.a + kStep * (2 * h + 1)]);
      const uint64_t vb = pack2(b[at.b + kStep * 2 * h], b[at.b + kStep * (2 * h + 1)]);
      f.ca[h] = at.turns ? fma2(vb, m, mul2(va, c)) : va;
      f.cb[h] = at.turns ? fma2(va, s, mul2(vb, c)) : vb;
    }
  }
}

// The normed and rotated head of a lane's eight values.  The whole warp calls.
template <int D, bool kInterleaved, bool kBias>
__device__ __forceinline__ Pairs turn(const uint4 &raw, const Factors &f, int norm, float eps, bool all_turn, bool turns) {
  constexpr int kLanes = D / 8;
  Pairs x = unpack<kInterleaved>(raw);
  float inv = 1.0f;
  if (norm != IDX_NORM_NONE) {
    float scale = 1.0f;
    for (;;) {
      float mean = 0.0f;
      Pairs d = x;
      if (kBias && norm == IDX_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) s += low(x.a[h]) + high(x.a[h]) + (low(x.b[h]) + high(x.b[h]));
        mean = group_sum<kLanes>(s) * (1.0f / D);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          d.a[h] = fma2(both(-mean), both(1.0f), x.a[h]);
          d.b[h] = fma2(both(-mean), both(1.0f), x.b[h]);
        }
      }
      uint64_t q = mul2(d.a[0], d.a[0]);
      q = fma2(d.a[1], d.a[1], q);
      q = fma2(d.b[0], d.b[0], q);
      q = fma2(d.b[1], d.b[1], q);
      const float s = group_sum<kLanes>(low(q) + high(q)) * (1.0f / D);
      // squares past fp32's range: once more with the head scaled down by 2^80, beside which
      // eps is nothing.  (A true infinity or NaN comes out the same way the second time.)
      const bool again = scale == 1.0f && !(s <= 3.402823466e38f);
      if (__any_sync(0xffffffffu, again)) {
        if (again) {
          scale = 0x1p-80f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            x.a[h] = mul2(x.a[h], both(scale));
            x.b[h] = mul2(x.b[h], both(scale));
          }
        }
        continue;
      }
      inv = rsqrtf(scale == 1.0f ? s + eps : s);
      x = d;
      break;
    }
  }
  Pairs z;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // where nothing turns, the other's factor is 0: an infinite other must not make it NaN
    const uint64_t oa = all_turn || turns ? x.b[h] : 0, ob = all_turn || turns ? x.a[h] : 0;
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
  __shared__ float2 cs[kMostRows][D / 2];
  __shared__ __align__(16) float weights[2][D], biases[kBias ? 2 : 1][kBias ? D : 1];   // of q and of k
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
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3, all_turn = p.rot == D;
  for (int unit = part * kWarps + warp; unit < rows * a.units; unit += a.splits * kWarps) {
    const int r = unit / a.units;
    int u = unit % a.units;
    const int64_t row = row0 + r;
    // the unit's kind and heads
    const int kind = u < a.q_units ? 0 : u < a.q_units + a.k_units ? 1 : 2;
    u -= kind == 0 ? 0 : kind == 1 ? a.q_units : a.q_units + a.k_units;
    const int h0 = u * a.heads, h_end = min(h0 + a.heads, kind == 0 ? p.Hq : p.Hkv);

    // the row's place in the cache
    bool live = false;
    char *to = nullptr;
    float *scale = nullptr;
    if (kind != 0 && p.slot != nullptr) {
      const uint32_t slot = static_cast<uint32_t>(p.slot[row]);   // negative slots are large ones
      live = slot < static_cast<uint64_t>(a.c.P) * kPage;
      const int64_t page = slot / kPage, tok = slot % kPage;
      to = static_cast<char *>(kind == 1 ? a.c.k : a.c.v) + (page * a.c.page_stride + tok * a.c.token_stride) * (f8 ? 1 : 2);
      scale = f8 ? (kind == 1 ? a.c.k_scale : a.c.v_scale) + page * p.Hkv * kPage + tok : nullptr;
    }

    if (kind == 2) {
      const uint16_t *const src = static_cast<const uint16_t *>(p.v) + row * p.v_stride + 8 * lane;
      uint4 raw[kVectors];
#pragma unroll
      for (int k = 0; k < kVectors; ++k) {
        const int h = h0 + k * kAtOnce + sub;
        raw[k] = make_uint4(0u, 0u, 0u, 0u);
        if (h < h_end) raw[k] = __ldcs(reinterpret_cast<const uint4 *>(src + h * D));
      }
#pragma unroll
      for (int k = 0; k < kVectors; ++k) {
        const int h = h0 + k * kAtOnce + sub;
        if (h0 + k * kAtOnce >= h_end) break;   // the warp's lanes together
        if (f8) {
          const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
          uint32_t lo, hi;
          const float sc = quantize(w, vector_amax<kLanes>(w), lo, hi);
          if (live && h < h_end) {
            *reinterpret_cast<uint2 *>(to + h * a.c.head_stride + 8 * lane) = make_uint2(lo, hi);
            if (lane == 0) scale[static_cast<int64_t>(h) * kPage] = sc;
          }
        } else if (live && h < h_end) {
          *reinterpret_cast<uint4 *>(to + (h * a.c.head_stride + 8 * lane) * 2) = raw[k];
        }
      }
      continue;
    }

    const uint16_t *const src = static_cast<const uint16_t *>(kind == 0 ? p.q : p.k) + row * (kind == 0 ? p.q_stride : p.k_stride);
    uint16_t *dst = static_cast<uint16_t *>(kind == 0 ? p.q_out : p.k_out);
    if (dst != nullptr) dst += row * (kind == 0 ? p.q_out_stride : p.k_out_stride);
    uint4 raw[kVectors];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
      const int h = h0 + k * kAtOnce + sub;
      raw[k] = make_uint4(0u, 0u, 0u, 0u);
      if (h < h_end) raw[k] = load<kInterleaved>(src + h * D, at);
    }
    Factors f;
    make_factors<kInterleaved, kBias>(at, cs[r], weights[kind], kBias ? biases[kind] : nullptr, f);
    const int norm = kind == 0 ? p.q_norm : p.k_norm;
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
      const int h = h0 + k * kAtOnce + sub;
      if (h0 + k * kAtOnce >= h_end) break;   // the warp's lanes together
      const bool here = h < h_end;
      const Pairs z = turn<D, kInterleaved, kBias>(raw[k], f, norm, p.eps, all_turn, at.turns);
      const uint4 out = pack<kInterleaved>(z);
      if (dst != nullptr && here) store<kInterleaved>(dst + h * D, at, out);
      if (to == nullptr) continue;
      if (!f8) {
        if (live && here) store<kInterleaved>(reinterpret_cast<uint16_t *>(to) + h * a.c.head_stride, at, out);
        continue;
      }
      // eight values in the order of their bytes
      const float v[8] = {low(z.a[0]), kInterleaved ? low(z.b[0]) : high(z.a[0]), kInterleaved ? high(z.a[0]) : low(z.a[1]),
                          kInterleaved ? high(z.b[0]) : high(z.a[1]), kInterleaved ? low(z.a[1]) : low(z.b[0]),
                          kInterleaved ? low(z.b[1]) : high(z.b[0]), kInterleaved ? high(z.a[1]) : low(z.b[1]), high(z.b[1])};
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
      uint32_t lo, hi;
      const float sc = quantize_f32(v, group_max<kLanes>(m), lo, hi);
      if (live && here) {
        char *const head = to + h * a.c.head_stride;
        if (kInterleaved) {
          *reinterpret_cast<uint2 *>(head + at.a) = make_uint2(lo, hi);
        } else {
          *reinterpret_cast<uint32_t *>(head + at.a) = lo;
          *reinterpret_cast<uint32_t *>(head + at.b) = hi;
        }
        if (lane == 0) scale[static_cast<int64_t>(h) * kPage] = sc;
      }
    }
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
