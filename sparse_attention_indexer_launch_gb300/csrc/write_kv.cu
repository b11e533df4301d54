// New tokens' keys and values into the paged cache.
//
// One vector of D values (a token's K or V of one head) is a group of D / 8 lanes
// with 16 bytes each: a vector is read once, its amax taken across the group by
// shuffles, and written once.  Memory bounds the call; each thread therefore has
// kVectors loads in flight before it needs the first.
#include <cuda_fp8.h>

#include "idx_device.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 4;   // vectors per group and pass

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {   // nearest codes, low byte a
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// E4M3 codes of the fp32 quotients f / sc.  x * (1 / sc) is within 3 * 2^-24 of the rounded
// quotient, so where the codes of that value times 1 - 2^-22 and 1 + 2^-22 agree they are
// the quotient's.  They disagree next to a tie only; those vectors, and scales out of the
// range where the reciprocal is exact to 2^-24, are divided.
__device__ __forceinline__ void quantize(const float (&f)[8], float sc, uint32_t &lo, uint32_t &hi) {
  const float inv = __frcp_rn(sc);
  const float down = inv * (1.0f - 0x1p-22f), up = inv * (1.0f + 0x1p-22f);
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = e4m3x2(f[2 * i] * down, f[2 * i + 1] * down);
    b[i] = e4m3x2(f[2 * i] * up, f[2 * i + 1] * up);
  }
  const bool same = a[0] == b[0] && a[1] == b[1] && a[2] == b[2] && a[3] == b[3];
  if (!(same && sc > 0x1p-100f && sc < 0x1p100f)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = e4m3x2(__fdiv_rn(f[2 * i], sc), __fdiv_rn(f[2 * i + 1], sc));
  }
  lo = a[0] | a[1] << 16;
  hi = a[2] | a[3] << 16;
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) write_kv_kernel(const WriteKvArgs a) {
  constexpr int kLanes = D / 8;               // lanes per vector
  constexpr int kGroups = kThreads / kLanes;  // vectors per CTA at a time
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const uint32_t per_row = 2u * a.c.Hkv;      // a row's K heads, then its V heads
  const int64_t tile0 = static_cast<int64_t>(blockIdx.x) * (kGroups * kVectors);
  const int64_t row0 = tile0 / per_row;
  const uint32_t rest0 = static_cast<uint32_t>(tile0 - row0 * per_row);
  uint4 x[kVectors];
  int32_t slot[kVectors];
  uint32_t part[kVectors];
#pragma unroll
  for (int u = 0; u < kVectors; ++u) {
    const uint32_t n = rest0 + u * kGroups + group;
    const int64_t r = row0 + n / per_row;
    slot[u] = -1;
    x[u] = make_uint4(0u, 0u, 0u, 0u);
    part[u] = n % per_row;
    if (r >= a.R) continue;
    slot[u] = a.slot[r];
    const bool is_v = part[u] >= static_cast<uint32_t>(a.c.Hkv);
    const uint32_t h = is_v ? part[u] - a.c.Hkv : part[u];
    const uint16_t *src = (is_v ? a.v_new : a.k_new) + r * a.row_stride + static_cast<int64_t>(h) * D;
    x[u] = __ldcs(reinterpret_cast<const uint4 *>(src) + lane);
  }
#pragma unroll
  for (int u = 0; u < kVectors; ++u) {
    const int64_t s = slot[u];
    const bool live = s >= 0 && s < a.c.P * kPage;
    const bool is_v = part[u] >= static_cast<uint32_t>(a.c.Hkv);
    const uint32_t h = is_v ? part[u] - a.c.Hkv : part[u];
    const int64_t page = s / kPage, tok = s % kPage;
    const int64_t at = page * a.c.page_stride + tok * a.c.token_stride + static_cast<int64_t>(h) * a.c.head_stride;
    if constexpr (!F8) {
      if (live) reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_v ? a.c.v : a.c.k) + at)[lane] = x[u];
    } else {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float f[8];
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
      }
      // every lane of the warp takes part, whether its vector is live or not
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float sc = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
      uint32_t lo, hi;
      quantize(f, sc, lo, hi);
      if (live) {
        reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? a.c.v : a.c.k) + at)[lane] = make_uint2(lo, hi);
        if (lane == 0) (is_v ? a.c.v_scale : a.c.k_scale)[(page * a.c.Hkv + h) * kPage + tok] = sc;
      }
    }
  }
}

template <int D, bool F8>
cudaError_t launch(const WriteKvArgs &a, cudaStream_t stream) {
  const int64_t per_cta = static_cast<int64_t>(kThreads / (D / 8)) * kVectors;
  const int64_t total = a.R * 2 * a.c.Hkv;
  write_kv_kernel<D, F8><<<static_cast<unsigned>((total + per_cta - 1) / per_cta), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_write_kv(const WriteKvArgs &a, cudaStream_t stream) {
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3;
  if (a.c.D == 64) return f8 ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
  return f8 ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
}

}  // namespace idx
