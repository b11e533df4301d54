// Norms of queries and keys for each head, their rotation, and keys and values into the
// paged cache, in one pass over a projection's output.
//
// A vector of D values (one head of a row) is a group of D / 8 lanes with 16 bytes each,
// read once and written once.  A warp takes heads of one row and one kind (q, k or v), so
// that the row's angles are worked out once for all of them.  The rotation is linear in
// the normed head, y = inv * (x - mean) * w + b, so weight, bias, cosine and sine fold into
// three factors per element before the loop over heads:
//     z = inv * ((x - mean) A + (x' - mean) B) + C,
// with x' the element that x turns with (another lane's for halves, the same lane's for
// interleaved pairs).
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
constexpr int kVectors = 4;   // loads of a lane in flight

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
  // half turns in [-1, 1): 32 of the 64 bits, rounded to fp32 relative to their own size
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &s, &c);
  if (!(fabsf(inv_freq) <= 3.402823466e38f)) s = c = __int_as_float(0x7FFFFFFF);   // no angle
  return make_float2(c, s);
}

__device__ __forceinline__ void unpack(const uint4 &v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = reinterpret_cast<const uint32_t &>(p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
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

// Eight values at p (32-byte steps from an aligned array), or eight times `otherwise`.
__device__ __forceinline__ void load8(const float *p, float otherwise, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 v = p != nullptr ? reinterpret_cast<const float4 *>(p)[i]
                                  : make_float4(otherwise, otherwise, otherwise, otherwise);
    x[4 * i] = v.x;
    x[4 * i + 1] = v.y;
    x[4 * i + 2] = v.z;
    x[4 * i + 3] = v.w;
  }
}

// The head's factors of a lane's eight elements, and the lane that holds their partners.
struct Factors {
  float a[8], b[8], c[8];
  int partner;     // halves: lane of the warp; interleaved: unused
  bool turns;      // the lane's dimensions are rotated
};

template <int D, bool kInterleaved>
__device__ __forceinline__ void make_factors(const idx_norm_rope_args &p, const float2 *cs, const float *weight,
                                             const float *bias, Factors &f) {
  constexpr int kLanes = D / 8;
  const int lane = threadIdx.x % kLanes, e0 = 8 * lane, half = p.rot >> 1;
  f.turns = e0 < p.rot;
  const bool second = !kInterleaved && e0 >= half;          // the pair's b, with a half before it
  const int q0 = !f.turns || kInterleaved ? e0 : second ? e0 - half : e0 + half;   // the partners' first element
  f.partner = (threadIdx.x & 31) - lane + q0 / 8;
  float w[8], wq[8], b[8], bq[8];
  load8(weight != nullptr ? weight + e0 : nullptr, 1.0f, w);
  load8(bias != nullptr ? bias + e0 : nullptr, 0.0f, b);
  if constexpr (kInterleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      wq[j] = w[j ^ 1];
      bq[j] = b[j ^ 1];
    }
  } else {
    load8(weight != nullptr ? weight + q0 : nullptr, 1.0f, wq);
    load8(bias != nullptr ? bias + q0 : nullptr, 0.0f, bq);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float2 t = make_float2(1.0f, 0.0f);
    if (f.turns) t = kInterleaved ? cs[(e0 + j) >> 1] : cs[(second ? e0 - half : e0) + j];
    const float sn = (kInterleaved ? (j & 1) != 0 : second) ? t.y : -t.y;
    f.a[j] = w[j] * t.x;
    f.b[j] = wq[j] * sn;
    // -0 adds nothing to any value, a zero's sign included
    f.c[j] = bias == nullptr ? -0.0f : f.turns ? b[j] * t.x + bq[j] * sn : b[j];
  }
}

// The normed and rotated head z of a lane's eight elements.  The whole warp calls.
template <int D, bool kInterleaved>
__device__ __forceinline__ void turn(const uint4 &raw, const Factors &f, int norm, float eps, float (&z)[8]) {
  constexpr int kLanes = D / 8;
  float x[8], y[8];
  unpack(raw, x);
  if constexpr (kInterleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
  } else {
    uint4 other;
    other.x = __shfl_sync(0xffffffffu, raw.x, f.partner);
    other.y = __shfl_sync(0xffffffffu, raw.y, f.partner);
    other.z = __shfl_sync(0xffffffffu, raw.z, f.partner);
    other.w = __shfl_sync(0xffffffffu, raw.w, f.partner);
    unpack(other, y);
  }
  float inv = 1.0f;
  if (norm != IDX_NORM_NONE) {
    float scale = 1.0f;
    for (;;) {
      float mean = 0.0f;
      if (norm == IDX_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s += x[j];
        mean = group_sum<kLanes>(s) * (1.0f / D);
      }
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = x[j] - mean;
        s = fmaf(d, d, s);
      }
      s = group_sum<kLanes>(s) * (1.0f / D);
      // squares past fp32's range: once more with the head scaled down by 2^80, beside which
      // eps is nothing.  (A true infinity or NaN comes out the same way the second time.)
      const bool again = scale == 1.0f && !(s <= 3.402823466e38f);
      if (__any_sync(0xffffffffu, again)) {
        if (again) {
          scale = 0x1p-80f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] *= scale;
            y[j] *= scale;
          }
        }
        continue;
      }
      inv = rsqrtf(scale == 1.0f ? s + eps : s);
      if (norm == IDX_NORM_LAYER) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] -= mean;
          y[j] -= mean;
        }
      }
      break;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // where nothing turns, B is 0: an infinite partner must not make it NaN
    const float t = f.turns ? fmaf(x[j], f.a[j], y[j] * f.b[j]) : x[j] * f.a[j];
    z[j] = fmaf(inv, t, f.c[j]);
  }
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  __shared__ float2 cs_all[kWarps][D / 2];
  const idx_norm_rope_args &p = a.p;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x % 32 / kLanes, warp = threadIdx.x / 32;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t row = unit / a.jobs;
  if (row >= p.R || (p.rows != nullptr && row >= *p.rows)) return;
  int job = static_cast<int>(unit % a.jobs);
  // the job's kind and heads
  const int kind = job < a.q_jobs ? 0 : job < a.q_jobs + a.k_jobs ? 1 : 2;
  job -= kind == 0 ? 0 : kind == 1 ? a.q_jobs : a.q_jobs + a.k_jobs;
  const int h0 = job * a.heads, h_end = min(h0 + a.heads, kind == 0 ? p.Hq : p.Hkv);
  const uint16_t *const src = static_cast<const uint16_t *>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                              row * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride) + lane * 8;
  uint16_t *dst = static_cast<uint16_t *>(kind == 0 ? p.q_out : kind == 1 ? p.k_out : nullptr);
  if (dst != nullptr) dst += row * (kind == 0 ? p.q_out_stride : p.k_out_stride) + lane * 8;

  // the row's place in the cache
  bool live = false;
  char *to = nullptr;
  float *scale = nullptr;
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3;
  if (kind != 0 && p.slot != nullptr) {
    const uint32_t slot = static_cast<uint32_t>(p.slot[row]);   // negative slots are large ones
    live = slot < static_cast<uint64_t>(a.c.P) * kPage;
    const int64_t page = slot / kPage, tok = slot % kPage;
    to = static_cast<char *>(kind == 1 ? a.c.k : a.c.v) +
         (page * a.c.page_stride + tok * a.c.token_stride + lane * 8) * (f8 ? 1 : 2);
    scale = f8 ? (kind == 1 ? a.c.k_scale : a.c.v_scale) + page * p.Hkv * kPage + tok : nullptr;
  }

  Factors f;
  if (kind != 2) {
    const int pairs = p.rot >> 1;
    for (int i = threadIdx.x % 32; i < pairs; i += 32)
      cs_all[warp][i] = cos_sin(p.pos[p.axis[i] * p.pos_stride + row], p.inv_freq[i]);
    __syncwarp();
    make_factors<D, kInterleaved>(p, cs_all[warp], kind == 0 ? p.q_weight : p.k_weight,
                                  kind == 0 ? p.q_bias : p.k_bias, f);
  }
  const int norm = kind == 0 ? p.q_norm : p.k_norm;

  for (int hb = h0; hb < h_end; hb += kVectors * kAtOnce) {
    uint4 raw[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const int h = hb + u * kAtOnce + sub;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h < h_end) raw[u] = *reinterpret_cast<const uint4 *>(src + h * D);
    }
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const int h = hb + u * kAtOnce + sub;
      if (hb + u * kAtOnce >= h_end) break;   // the warp's lanes together
      const bool here = h < h_end;
      uint32_t lo, hi;
      float sc;
      if (kind == 2) {
        if (f8) {
          const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
          sc = quantize(w, vector_amax<kLanes>(w), lo, hi);
        }
      } else {
        float z[8];
        turn<D, kInterleaved>(raw[u], f, norm, p.eps, z);
        if (to != nullptr && f8) {
          float m = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(z[j]));
          sc = quantize_f32(z, group_max<kLanes>(m), lo, hi);
        }
        raw[u] = pack_bf16(z);
        if (dst != nullptr && here) *reinterpret_cast<uint4 *>(dst + h * D) = raw[u];
      }
      if (live && here) {
        char *const at = to + h * a.c.head_stride * (f8 ? 1 : 2);
        if (f8) {
          *reinterpret_cast<uint2 *>(at) = make_uint2(lo, hi);
          if (lane == 0) scale[static_cast<int64_t>(h) * kPage] = sc;
        } else {
          *reinterpret_cast<uint4 *>(at) = raw[u];
        }
      }
    }
  }
}

template <int D, bool kInterleaved>
cudaError_t launch(NormRopeArgs a, int num_sms, cudaStream_t stream) {
  constexpr int kAtOnce = 32 / (D / 8);
  // heads of a warp: as many as keep the GPU full, so that few warps work out the same angles
  const int64_t vectors = a.p.R * (a.p.Hq + static_cast<int64_t>(a.p.Hkv) * (a.c.v != nullptr ? 2 : 1));
  const int64_t warps = static_cast<int64_t>(num_sms) * 32;
  int heads = kAtOnce;
  while (heads < 64 && vectors / (2 * heads) >= warps) heads *= 2;
  a.heads = heads;
  a.q_jobs = (a.p.Hq + heads - 1) / heads;
  a.k_jobs = (a.p.Hkv + heads - 1) / heads;
  a.jobs = a.q_jobs + a.k_jobs * (a.c.v != nullptr ? 2 : 1);
  const int64_t grid = (a.p.R * a.jobs + kWarps - 1) / kWarps;
  norm_rope_kernel<D, kInterleaved><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, int num_sms, cudaStream_t stream) {
  const bool il = a.p.interleaved != 0;
  if (a.p.D == 64) return il ? launch<64, true>(a, num_sms, stream) : launch<64, false>(a, num_sms, stream);
  if (a.p.D == 128) return il ? launch<128, true>(a, num_sms, stream) : launch<128, false>(a, num_sms, stream);
  return il ? launch<256, true>(a, num_sms, stream) : launch<256, false>(a, num_sms, stream);
}

}  // namespace idx
