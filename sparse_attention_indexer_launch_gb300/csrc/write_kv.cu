// New tokens' keys and values into the paged cache.
//
// One vector of D values (a token's K or V of one head) is a group of D / 8 lanes
// with 16 bytes each: a vector is read once, its amax taken across the group by
// shuffles, and written once.  The grid's groups walk the rows in steps of a whole
// number of rows, so a group keeps its head (K or V, pointers, scale offset) for the
// whole call and an address costs it two multiplications by the slot's page and
// token; kVectors loads are in flight before the first is needed.  In E4M3 the call
// is bound by instructions as much as by memory: what a vector costs beyond its loads
// is kept small (amax in packed bf16, quotients by a two-term reciprocal).  Measured: 61,084
// tokens x 8 heads of 128 dimensions into E4M3 73.6 us, 5.2 TB/s; into bf16 82.5 us, 6.1
// TB/s; 32 tokens 5.4 us, what the host needs for a call.
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

__device__ __forceinline__ uint64_t pack2(float x, float y) {
  return static_cast<uint64_t>(__float_as_uint(y)) << 32 | __float_as_uint(x);
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t z;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  return z;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t w) {
  uint64_t z;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(z) : "l"(x), "l"(y), "l"(w));
  return z;
}

// The scale amax / 448 and the E4M3 codes of the quotients x / scale, both as fp32
// division rounds them.  A divisor's reciprocal in two terms, hi + lo, gives
// x / d = fma(x, hi, x * lo) correctly rounded (Brisebarre and Muller's multiplication by
// a constant of higher precision): bf16 significands have 8 bits, and all 128 x 128 pairs
// of amax and x were compared with the division, for every hi within 3 units of the last
// place.  A single product would not do: 3/4 of the amax, for one, lies on a tie between
// two codes.  Amaxes near the ends of the range, zero and infinity take the division.
__device__ __forceinline__ float quantize(const uint32_t (&w)[4], float amax, uint32_t &lo, uint32_t &hi) {
  float sc;
  uint32_t c[4];
  if (amax > 0x1p-100f && amax < 0x1p100f) {
    constexpr float kHi = 0x1.24924ap-9f, kLo = -0x1.b6db6ep-34f;   // 1 / 448
    sc = fmaf(amax, kHi, amax * kLo);
    const float r = __fdividef(1.0f, sc);
    const float e = fmaf(-r, sc, 1.0f) * r;
    const uint64_t r2 = pack2(r, r), e2 = pack2(e, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t f = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      const uint64_t q = fma2(f, r2, mul2(f, e2));
      c[i] = e4m3x2(__uint_as_float(static_cast<uint32_t>(q)), __uint_as_float(static_cast<uint32_t>(q >> 32)));
    }
  } else {
    sc = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3x2(__fdiv_rn(__uint_as_float(w[i] << 16), sc), __fdiv_rn(__uint_as_float(w[i] & 0xFFFF0000u), sc));
  }
  lo = c[0] | c[1] << 16;
  hi = c[2] | c[3] << 16;
  return sc;
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

  // the warp stays together while any of its groups has rows left
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
        // exact in bf16: a maximum rounds nothing (NaN is passed over, as the indexer's new keys do)
        __nv_bfloat162 m = __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[0]));
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[i])));
        // every lane of the warp takes part, whether its vector is live or not
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float amax = fmaxf(__low2float(m), __high2float(m));
        uint32_t lo, hi;
        const float sc = quantize(w, amax, lo, hi);
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
