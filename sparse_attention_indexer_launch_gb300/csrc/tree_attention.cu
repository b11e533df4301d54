// Attention of drafted tokens over a paged cache, whole or at selected positions.
//
// One CTA takes eight query heads (fewer where a key head serves fewer) of one row
// and walks the row's positions: the cached ones (all, or the row's selection), then
// the drafted tokens of its mask.  A warp takes every eighth position with its
// dimensions spread over the lanes, and keeps each head's running maximum, sum and
// output (the softmax in one pass); the eight warps' results are joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "idx_device.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr int kWarps = 8;
constexpr int kHeadsPerCta = 8;

template <int D, bool F8>
__global__ void __launch_bounds__(kWarps * 32) tree_attention_kernel(const TreeAttnArgs a) {
  constexpr int E = D / 32;   // dimensions per lane: lane * E ..
  const idx_tree_problem &p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.Hq / p.cache.Hkv;
  const int r = blockIdx.x;
  const int h = blockIdx.y;                       // key/value head
  const int g0 = blockIdx.z * kHeadsPerCta;       // first query head of the group
  const int ng = min(kHeadsPerCta, G - g0);
  // the row's request
  int lo = 0, hi = p.Q;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.row_start[mid] <= r) lo = mid;
    else hi = mid;
  }
  const int i = lo;
  const int rs = p.row_start[i], re = p.row_start[i + 1];
  if (r < rs || r >= re) return;
  uint32_t bad = 0;
  if (rs < 0 || re > p.R || re - rs > p.max_new) bad |= kStatusBadBound;
  const int T = min(re - rs, p.max_new);
  const int t = r - rs;
  if (rs < 0 || re > p.R || t >= T) {   // rows past the host's bound are not written
    flag_status(a.status, kStatusBadBound);
    return;
  }
  int ctx = p.ctx_len[i];
  if (ctx < 0 || ctx > p.max_ctx) bad |= kStatusBadBound;
  ctx = max(0, min(ctx, p.max_ctx));
  const int64_t room = static_cast<int64_t>(p.pt_stride) * kPage;
  if (ctx + T > room) bad |= kStatusBadBound;
  const uint64_t mask = p.mask != nullptr ? p.mask[r] : (2ull << t) - 1ull;
  const int nctx = a.sel != nullptr ? a.sel_k : ctx;
  float q[kHeadsPerCta][E], o[kHeadsPerCta][E], m[kHeadsPerCta], l[kHeadsPerCta];
  const uint16_t *qr = static_cast<const uint16_t *>(p.q) + static_cast<int64_t>(r) * p.q_row_stride +
                       static_cast<int64_t>(h * G + g0) * D + lane * E;
#pragma unroll
  for (int g = 0; g < kHeadsPerCta; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[g][e] = g < ng ? __uint_as_float(static_cast<uint32_t>(qr[g * D + e]) << 16) * p.scale : 0.0f;
      o[g][e] = 0.0f;
    }
  }
  for (int n = warp; n < nctx + T; n += kWarps) {
    int64_t j;
    if (n < nctx) {
      j = n;
      if (a.sel != nullptr) {
        j = a.sel[static_cast<int64_t>(r) * a.sel_k + n];
        if (j < 0 || j >= ctx) continue;
      }
    } else {
      if (!((mask >> (n - nctx)) & 1ull)) continue;
      j = ctx + (n - nctx);
    }
    if (j >= room) continue;
    const int32_t page = p.page_table[static_cast<int64_t>(i) * p.pt_stride + j / kPage];
    if (page < 0 || page >= p.cache.P) {
      bad |= kStatusBadPage;
      continue;
    }
    const int64_t at = page * p.cache.page_stride + (j % kPage) * p.cache.token_stride + h * p.cache.head_stride + lane * E;
    float k[E], v[E], ks = 1.0f, vs = 1.0f;
    if constexpr (F8) {
      const int64_t sat = (static_cast<int64_t>(page) * p.cache.Hkv + h) * kPage + j % kPage;
      ks = p.cache.k_scale[sat];
      vs = p.cache.v_scale[sat];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (F8) {
        k[e] = static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(p.cache.k)[at + e]);
        v[e] = static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(p.cache.v)[at + e]) * vs;
      } else {
        k[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.cache.k)[at + e]);
        v[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.cache.v)[at + e]);
      }
    }
#pragma unroll
    for (int g = 0; g < kHeadsPerCta; ++g) {
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) s += q[g][e] * k[e];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= ks;
      const float nm = fmaxf(m[g], s);
      const float keep = m[g] == nm ? 1.0f : __expf(m[g] - nm), pr = __expf(s - nm);
      m[g] = nm;
      l[g] = l[g] * keep + pr;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = o[g][e] * keep + pr * v[e];
    }
  }
  __shared__ float sm[kWarps][kHeadsPerCta], sl[kWarps][kHeadsPerCta], so[kWarps][D];
  if (lane == 0)
    for (int g = 0; g < kHeadsPerCta; ++g) {
      sm[warp][g] = m[g];
      sl[warp][g] = l[g];
    }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < kHeadsPerCta; ++g) {
    if (g >= ng) break;
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w][g]);
    for (int w = 0; w < kWarps; ++w) sum += sl[w][g] > 0.0f || isnan(sl[w][g]) ? sl[w][g] * __expf(sm[w][g] - top) : 0.0f;
    const float mine = m[g] == -INFINITY ? 0.0f : __expf(m[g] - top);
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = l[g] == 0.0f ? 0.0f : o[g][e] * mine;
    __syncthreads();
    const int64_t head = static_cast<int64_t>(r) * p.Hq + h * G + g0 + g;
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
      float acc = 0.0f;
      for (int w = 0; w < kWarps; ++w) acc += so[w][d];
      reinterpret_cast<__nv_bfloat16 *>(a.out)[head * D + d] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc / sum);
    }
    if (threadIdx.x == 0 && a.lse != nullptr) a.lse[head] = sum == 0.0f ? -INFINITY : top + __logf(sum);
    __syncthreads();
  }
  if (bad) flag_status(a.status, bad);
}

}  // namespace

cudaError_t launch_tree_attention(const TreeAttnArgs &a, int, cudaStream_t stream) {
  const int G = a.p.Hq / a.p.cache.Hkv;
  const dim3 grid(a.p.R, a.p.cache.Hkv, (G + kHeadsPerCta - 1) / kHeadsPerCta);
  const bool f8 = a.p.cache.kv_dtype == IDX_KV_E4M3;
  if (a.p.cache.D == 64) {
    if (f8) tree_attention_kernel<64, true><<<grid, kWarps * 32, 0, stream>>>(a);
    else tree_attention_kernel<64, false><<<grid, kWarps * 32, 0, stream>>>(a);
  } else {
    if (f8) tree_attention_kernel<128, true><<<grid, kWarps * 32, 0, stream>>>(a);
    else tree_attention_kernel<128, false><<<grid, kWarps * 32, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace idx
