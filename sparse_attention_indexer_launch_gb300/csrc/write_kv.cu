// New tokens' keys and values into the paged cache.
//
// One vector of D values (a token's K or V of one head) is a group of D / 8 lanes
// with 16 bytes each: a vector is read once, its amax taken across the group by
// shuffles, and written once.  The grid's groups walk the rows in steps of a whole
// number of rows, so a group keeps its head (K or V, pointers, scale offset) for the
// whole call and an address costs it two multiplications by the slot's page and
// token; kVectors loads are in flight before the first is needed.  In E4M3 the call
// is bound by instructions as much as by memory: what a vector costs beyond its loads
// is kept small (amax in packed bf16, quotients by a checked reciprocal).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "idx_device.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 4;    // vectors per group and pass
constexpr int kCtasPerSm = 5;  // 48 registers a thread hold four loads; all CTAs are resident

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {   // nearest codes, low byte a
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// E4M3 codes of the fp32 quotients f / sc.  x times an approximate reciprocal (within
// 2^-23) is within 2^-22 of the rounded quotient, so where the codes of that value
// times 1 - 2^-21 and 1 + 2^-21 agree they are the quotient's.  They disagree next to a
// tie only; those vectors, and scales near the ends of the range, are divided.
__device__ __forceinline__ void quantize(const uint32_t (&w)[4], float sc, uint32_t &lo, uint32_t &hi) {
  const float inv = __fdividef(1.0f, sc);
  const float down = inv * (1.0f - 0x1p-21f), up = inv * (1.0f + 0x1p-21f);
  uint32_t a[4], b[4];
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    a[i] = e4m3x2(f[2 * i] * down, f[2 * i + 1] * down);
    b[i] = e4m3x2(f[2 * i] * up, f[2 * i + 1] * up);
  }
  lo = a[0] | a[1] << 16;
  hi = a[2] | a[3] << 16;
  const bool same = lo == (b[0] | b[1] << 16) && hi == (b[2] | b[3] << 16);
  if (!(same && sc > 0x1p-100f && sc < 0x1p100f)) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {   // rare: kept small
      const float *const g = f + 4 * i;
      const uint32_t c = e4m3x2(__fdiv_rn(g[0], sc), __fdiv_rn(g[1], sc)) |
                         e4m3x2(__fdiv_rn(g[2], sc), __fdiv_rn(g[3], sc)) << 16;
      if (i == 0) lo = c;
      else hi = c;
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) write_kv_kernel(const WriteKvArgs a) {
  constexpr int kLanes = D / 8;               // lanes per vector
  constexpr int kGroups = kThreads / kLanes;  // vectors per CTA at a time
  const int lane = threadIdx.x % kLanes;
  const uint32_t per_row = 2u * a.c.Hkv;      // a row's K heads, then its V heads
  const uint32_t group = blockIdx.x * kGroups + threadIdx.x / kLanes;
  const uint32_t rows_at_once = gridDim.x * kGroups / per_row;   // at least 1: see launch()
  const uint32_t part = group % per_row;
  const bool is_v = part >= static_cast<uint32_t>(a.c.Hkv);
  const uint32_t h = is_v ? part - a.c.Hkv : part;
  // groups past the last whole row have nothing to do, but take part in the shuffles
  int64_t row = group < rows_at_once * per_row ? group / per_row : a.R;
  const uint16_t *const src = (is_v ? a.v_new : a.k_new) + static_cast<int64_t>(h) * D + lane * 8;
  constexpr int kBytes = F8 ? 1 : 2;
  char *const dst = static_cast<char *>(is_v ? a.c.v : a.c.k) + (static_cast<int64_t>(h) * a.c.head_stride + lane * 8) * kBytes;
  float *const scale = F8 ? (is_v ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(h) * kPage : nullptr;
  const uint32_t limit = static_cast<uint32_t>(min(a.c.P * kPage, static_cast<int64_t>(INT32_MAX)));   // slots

  // the warp stays together: its first row decides
  while (__any_sync(0xffffffffu, row < a.R)) {
    uint4 x[kVectors];
    uint32_t slot[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const int64_t r = row + static_cast<int64_t>(u) * rows_at_once;
      slot[u] = ~0u;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < a.R) {
        slot[u] = static_cast<uint32_t>(a.slot[r]);
        x[u] = __ldcs(reinterpret_cast<const uint4 *>(src + r * a.row_stride));
      }
    }
    row += static_cast<int64_t>(kVectors) * rows_at_once;
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const bool live = slot[u] < limit;   // negative slots are large ones
      const uint32_t page = slot[u] / kPage, tok = slot[u] % kPage;
      char *const to = dst + (page * a.c.page_stride + tok * a.c.token_stride) * kBytes;
      if constexpr (!F8) {
        if (live) *reinterpret_cast<uint4 *>(to) = x[u];
      } else {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        // exact in bf16: a maximum rounds nothing (NaN is passed over)
        __nv_bfloat162 m = __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[0]));
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[i])));
        // every lane of the warp takes part, whether its vector is live or not
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float amax = fmaxf(__low2float(m), __high2float(m));
        const float sc = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
        uint32_t lo, hi;
        quantize(w, sc, lo, hi);
        if (live) {
          *reinterpret_cast<uint2 *>(to) = make_uint2(lo, hi);
          if (lane == 0) scale[static_cast<int64_t>(page) * a.c.Hkv * kPage + tok] = sc;
        }
      }
    }
  }
}

template <int D, bool F8>
cudaError_t launch(const WriteKvArgs &a, int num_sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  // one vector per group while the GPU holds them all at once, walks of several beyond;
  // never less than a row
  const int64_t per_row = 2 * static_cast<int64_t>(a.c.Hkv);
  const int64_t most = std::max(static_cast<int64_t>(kCtasPerSm) * num_sms, (per_row + kGroups - 1) / kGroups);
  const int64_t all = (a.R * per_row + kGroups - 1) / kGroups;
  write_kv_kernel<D, F8><<<static_cast<unsigned>(std::min(all, most)), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_write_kv(const WriteKvArgs &a, int num_sms, cudaStream_t stream) {
  const bool f8 = a.c.kv_dtype == IDX_KV_E4M3;
  if (a.c.D == 64) return f8 ? launch<64, true>(a, num_sms, stream) : launch<64, false>(a, num_sms, stream);
  return f8 ? launch<128, true>(a, num_sms, stream) : launch<128, false>(a, num_sms, stream);
}

}  // namespace idx
