// E4M3 vectors of the key/value cache: the scale amax / 448 and the codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "idx_device.cuh"

namespace idx {

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

// The scale amax / 448 and the E4M3 codes of the quotients x / scale of a bf16 vector, both as fp32
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

// amax of a vector of bf16 pairs across its group of kLanes lanes (exact in bf16: a maximum
// rounds nothing; a NaN is passed over, as the indexer's new keys do).  The whole warp calls.
template <int kLanes>
__device__ __forceinline__ float vector_amax(const uint32_t (&w)[4]) {
  __nv_bfloat162 m = __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[0]));
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[i])));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return fmaxf(__low2float(m), __high2float(m));
}

// The same of eight fp32 values a lane.  The two-term reciprocal gives each quotient to within
// an fp32 rounding or so of the division's; a code can differ from the division's only where
// that quotient lies within it of a tie.
__device__ __forceinline__ float quantize_f32(const float (&x)[8], float amax, uint32_t &lo, uint32_t &hi) {
  float sc;
  uint32_t c[4];
  if (amax > 0x1p-100f && amax < 0x1p100f) {
    sc = __fdiv_rn(amax, 448.0f);
    const float r = __fdividef(1.0f, sc);
    const float e = fmaf(-r, sc, 1.0f) * r;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(fmaf(x[2 * i], r, x[2 * i] * e), fmaf(x[2 * i + 1], r, x[2 * i + 1] * e));
  } else {
    sc = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-149f) : 1.0f;   // 0 would leave 0 / 0
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(__fdiv_rn(x[2 * i], sc), __fdiv_rn(x[2 * i + 1], sc));
  }
  lo = c[0] | c[1] << 16;
  hi = c[2] | c[3] << 16;
  return sc;
}

}  // namespace idx
