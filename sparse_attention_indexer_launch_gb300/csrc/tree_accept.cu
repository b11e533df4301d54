// What a verify step keeps: the path through each request's drafted tree that the sampled
// tokens confirm, the pages behind it back on the free stack, and the accepted tokens' keys
// and values at consecutive positions.
//
// Acceptance walks down from token 0: the next token is the first child whose draft is the
// sampled token.  A warp holds a request's tree, two tokens a lane, so a step of the walk is
// two comparisons and a ballot.  Giving pages back needs a prefix sum over all requests'
// results: the CTA that finishes last does it, so nobody waits.  A single CTA, of a warp per
// request, has them in shared memory.  It is latency from end to end: 2.2 us in a graph for two
// requests, 6.5 for 1,024 trees (32 CTAs, the counter, then one CTA that sums 1,024 results, a
// request a thread, with the pages read before it is known to be the last one).  CTAs are as large as
// the batch, up to 1,024 threads, because a few requests in one of 1,024 were slower.
//
// Moving is in place: the a-th accepted token goes from the slot of row path[a] to that of row
// a, path[a] >= a and ascending.  Row a's slot is read by no later move (path[b] = a only for
// b <= a), so one group of lanes that takes a head's moves in order, loads ahead of stores,
// needs no copy.  Four loads a lane in flight: 512 requests of an E4M3 cache with up to five moves
// each 3.7 us in a graph where the bytes take 1.0; 8 requests 2.0, all launch.  Long paths go in rounds
// of four moves, path, slot and data one after the other: 62 moves in each of 8 requests 18.7 us (bytes
// 0.3), of 512 27.5 us (19.8; bf16 44.1 for 38.4).
#include <algorithm>

#include "idx_device.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr int kWalkThreads = 1024;   // at most: a request per warp, and per thread where pages go back
constexpr int kWalkWarps = kWalkThreads / 32;
constexpr int kThreads = 256;
constexpr int kMoves = 4;   // loads of a lane in flight

__device__ __forceinline__ int32_t pages_of(int64_t tokens) {
  return static_cast<int32_t>((tokens + kPage - 1) / kPage);
}

// Rows of request i: first and number, with the array's ends kept whatever it holds.
__device__ __forceinline__ void rows_of(const int32_t *row_start, int i, int32_t cap, int32_t &first, int32_t &n, uint32_t &bad) {
  const int32_t a = row_start[i], b = row_start[i + 1];
  first = min(max(a, 0), cap);
  n = min(max(b, first), cap) - first;
  if (first != a || static_cast<int64_t>(first) + n != b) bad |= kStatusBadBound;
}

// A request's cached tokens, its pages [first, end) of which the last may go back, two of them read.
struct Held {
  int32_t ctx, first, end, page[2];
};
__device__ __forceinline__ Held held_by(const idx_tree_accept_args &t, int i) {
  uint32_t bad = 0;   // recorded where the request is walked
  int32_t row, n;
  rows_of(t.row_start, i, t.cap, row, n, bad);
  Held h;
  h.ctx = min(max(t.ctx_len[i], 0), (1 << 30) - kPage);
  h.first = pages_of(static_cast<int64_t>(h.ctx) + min(n, 1));   // token 0 stays
  h.end = min(pages_of(static_cast<int64_t>(h.ctx) + n), t.pt_stride);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    h.page[k] = h.first + k < h.end ? t.page_table[static_cast<int64_t>(i) * t.pt_stride + h.first + k] : -1;
  return h;
}

__global__ void __launch_bounds__(kWalkThreads, 1) tree_accept_kernel(const TreeAcceptArgs a) {
  __shared__ int32_t warp_pages[kWalkWarps], lengths[kWalkWarps];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
  const idx_tree_accept_args &t = a.t;
  uint32_t bad = 0;
  grid_dependency_trigger();
  grid_dependency_wait();

  for (int i = blockIdx.x * warps + warp; i < t.Q; i += gridDim.x * warps) {
    int32_t first, n;
    rows_of(t.row_start, i, t.cap, first, n, bad);
    if (n > IDX_MAX_TREE) bad |= kStatusBadBound;
    const int32_t tree = min(n, IDX_MAX_TREE);
    // tokens `lane` and `lane + 32`; token 0 and those without an earlier parent are nobody's children
    int32_t parent[2], draft[2], target[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = lane + 32 * k;
      parent[k] = -1;
      draft[k] = target[k] = 0;
      if (u < tree) {
        draft[k] = t.draft[first + u];
        target[k] = t.target[first + u];
        parent[k] = t.parent != nullptr ? t.parent[first + u] : u - 1;
        if (parent[k] >= u || parent[k] < -1) {
          bad |= kStatusBadBound;
          parent[k] = -1;
        }
      }
    }
    int node = 0, length = tree > 0 ? 1 : 0;
    int32_t next = tree > 0 ? __shfl_sync(0xffffffffu, target[0], 0) : -1;
    int32_t mine[2] = {lane == 0 && tree > 0 ? 0 : -1, -1};   // accepted tokens `lane` and `lane + 32`
    int32_t token[2] = {lane == 0 ? next : -1, -1};
    while (length > 0 && length < tree) {
      const uint32_t lo = __ballot_sync(0xffffffffu, parent[0] == node && draft[0] == next);
      const uint32_t hi = __ballot_sync(0xffffffffu, parent[1] == node && draft[1] == next);
      if ((lo | hi) == 0) break;
      node = lo != 0 ? __ffs(lo) - 1 : 31 + __ffs(hi);
      next = __shfl_sync(0xffffffffu, lo != 0 ? target[0] : target[1], node & 31);
      if (length == lane) {
        mine[0] = node;
        token[0] = next;
      } else if (length == lane + 32) {
        mine[1] = node;
        token[1] = next;
      }
      ++length;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (lane + 32 * k < tree) {
        t.path[first + lane + 32 * k] = mine[k];
        t.token[first + lane + 32 * k] = token[k];
      }
    }
    for (int u = IDX_MAX_TREE + lane; u < n; u += 32) t.path[first + u] = t.token[first + u] = -1;
    if (lane == 0) {
      t.accept_len[i] = length;
      lengths[warp] = length;
      t.last[i] = next;
    }
  }
  if (bad) flag_status(a.status, bad);

  // What giving pages back needs beside the lengths is read by every CTA before it is known which
  // one comes last: a request's rows and cached tokens, and its pages from the first that may go.
  Held held{};
  if (tid < t.Q) held = held_by(t, tid);

  // the CTA that comes last sees every request's length
  const bool alone = gridDim.x == 1 && t.Q <= warps;
  if (!alone) {
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(a.arrived, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (tid == 0) *a.arrived = 0;
  } else {
    __syncthreads();
  }
  bad = 0;
  const int32_t had = max(*t.free_count, 0);
  int64_t base = had;
  for (int i0 = 0; i0 < t.Q; i0 += threads) {
    const int i = i0 + tid;
    int32_t keep = 0, have = 0;   // the first page behind the new length, those from there on with an id
    if (i0 > 0 && i < t.Q) held = held_by(t, i);
    const auto page_at = [&](int32_t p) {
      const int32_t k = p - held.first;
      return k == 0 ? held.page[0] : k == 1 ? held.page[1] : t.page_table[static_cast<int64_t>(i) * t.pt_stride + p];
    };
    if (i < t.Q) {
      const int32_t length = alone ? lengths[i] : __ldcg(t.accept_len + i);
      keep = pages_of(static_cast<int64_t>(held.ctx) + length);
      for (int32_t p = keep; p < held.end; ++p) {
        const int32_t page = page_at(p);
        if (page >= 0 && page < t.P) ++have;
        else bad |= kStatusBadPage;
      }
      t.new_ctx[i] = held.ctx + length;
    }
    int32_t upto = have;   // places on the stack: a prefix sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    if (lane == 31) warp_pages[warp] = upto;
    __syncthreads();
    int64_t before = base + upto - have;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += warp_pages[w];
      base += warp_pages[w];
    }
    for (int32_t p = keep; i < t.Q && p < held.end; ++p) {
      const int32_t page = page_at(p);
      if (page < 0 || page >= t.P) continue;
      if (before < t.free_cap) t.free_pages[before] = page;
      else bad |= kStatusBadPage;
      ++before;
    }
    __syncthreads();
  }
  if (tid == 0) *t.free_left = static_cast<int32_t>(min(base, static_cast<int64_t>(t.free_cap)));
  if (bad) flag_status(a.status, bad);
}

// One group of D * bytes / 16 lanes moves one head's keys or values of one request.
template <int kLanes>
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const TreeCommitArgs a) {
  const int lane = threadIdx.x % kLanes;
  grid_dependency_trigger();
  const int64_t group = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
  const int per_req = a.c.Hkv * (a.c.v != nullptr ? 2 : 1);
  const int64_t i = group / per_req;
  if (i >= a.Q) return;
  int h = static_cast<int>(group % per_req);
  const bool is_v = h >= a.c.Hkv;
  if (is_v) h -= a.c.Hkv;
  uint32_t bad = 0;
  int32_t first, n;
  grid_dependency_wait();
  rows_of(a.row_start, static_cast<int>(i), a.cap, first, n, bad);
  const int32_t length = min(a.accept_len[i], min(n, IDX_MAX_TREE));
  const int bytes = a.c.kv_dtype == IDX_KV_E4M3 ? 1 : 2;
  char *const base = static_cast<char *>(is_v ? a.c.v : a.c.k) + h * a.c.head_stride * bytes + lane * 16;
  float *const scale = bytes == 1 ? (is_v ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(h) * kPage : nullptr;
  const uint32_t limit = static_cast<uint32_t>(a.c.P * kPage);
  const auto place = [&](uint32_t slot) { return (slot / kPage * a.c.page_stride + slot % kPage * a.c.token_stride) * bytes; };
  const auto scale_at = [&](uint32_t slot) { return static_cast<int64_t>(slot / kPage) * a.c.Hkv * kPage + slot % kPage; };

  for (int t0 = 1; t0 < length; t0 += kMoves) {
    uint4 x[kMoves];
    float sc[kMoves];
    uint32_t to[kMoves];
#pragma unroll
    for (int k = 0; k < kMoves; ++k) {
      const int t = t0 + k;
      to[k] = ~0u;
      if (t >= length) continue;
      const int32_t from = a.path[first + t];
      if (from <= t || from >= n) continue;   // it is where it belongs (or no path)
      const uint32_t s = static_cast<uint32_t>(a.slot[first + from]), d = static_cast<uint32_t>(a.slot[first + t]);
      if (s >= limit || d >= limit) continue;   // negative slots are large ones
      to[k] = d;
      x[k] = *reinterpret_cast<const uint4 *>(base + place(s));
      if (scale != nullptr && lane == 0) sc[k] = scale[scale_at(s)];
    }
#pragma unroll
    for (int k = 0; k < kMoves; ++k) {
      if (to[k] == ~0u) continue;
      *reinterpret_cast<uint4 *>(base + place(to[k])) = x[k];
      if (scale != nullptr && lane == 0) scale[scale_at(to[k])] = sc[k];
    }
  }
}

template <int kLanes>
cudaError_t launch_commit(const TreeCommitArgs &a, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(a.Q) * a.c.Hkv * (a.c.v != nullptr ? 2 : 1) * kLanes;
  return launch_early(tree_commit_kernel<kLanes>, static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, 1, stream, a);
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptArgs &a, int num_sms, cudaStream_t stream) {
  const int warps = std::min(a.t.Q, kWalkWarps), grid = std::min((a.t.Q + warps - 1) / warps, 2 * num_sms);
  return launch_early(tree_accept_kernel, static_cast<unsigned>(grid), 32 * static_cast<unsigned>(warps), 0, 1, stream, a);
}

cudaError_t launch_tree_commit(const TreeCommitArgs &a, cudaStream_t stream) {
  const int lanes = a.c.D * (a.c.kv_dtype == IDX_KV_E4M3 ? 1 : 2) / 16;
  return lanes == 4 ? launch_commit<4>(a, stream) : lanes == 8 ? launch_commit<8>(a, stream) : launch_commit<16>(a, stream);
}

}  // namespace idx
