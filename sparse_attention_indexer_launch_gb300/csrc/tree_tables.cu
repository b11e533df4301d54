// Page tables, slot maps and tree masks of a step, from request lengths.
//
// Two prefix sums over the requests place everything: of new tokens (a row's
// request and token number) and of new pages (its place on the free stack).  With
// at most 4,096 requests a sum costs a CTA less than a second launch would, so
// every CTA does both in shared memory and then writes its own rows; no CTA waits
// for another.
//
// A row's page is read from the table only where the request held it before the
// call and taken from the free stack otherwise, so no CTA reads an entry that
// another one writes.
//
// Long runs of rows are bound by instructions: four consecutive rows per thread take one
// lookup of the request (none while the last one's goes on) and one or two of a page.
// Measured: 4.0 million rows of 64 prompts 16.6 us, 3.9 TB/s of stores; 64 trees of up to 64
// tokens 8.2 us (the prefix sums and the walks up the trees); 2 x 4 rows 4.1 us, which is
// what the host needs for a call.
#include "idx_device.cuh"
#include "launch.h"

namespace idx {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 4;   // consecutive rows, so that a warp stores 512 bytes per array

// Lengths are the caller's data: cut to 2^30, which no cache holds, positions fit 31 bits.
constexpr int32_t kMaxLen = 1 << 30;
__device__ __forceinline__ int32_t length_of(int32_t n) { return min(max(n, 0), kMaxLen - kPage); }
// Pages that hold `tokens` tokens.
__device__ __forceinline__ int32_t pages_of(int32_t tokens) {
  return static_cast<int32_t>(static_cast<uint32_t>(tokens + kPage - 1) / kPage);
}

// Largest i in [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int find_last(const int32_t *v, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) tree_tables_kernel(const TreeTablesArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  int32_t *const start = reinterpret_cast<int32_t *>(smem_raw);   // rows before request i
  int32_t *const taken = start + a.t.Q + 1;                       // new pages before request i
  __shared__ int64_t warp_rows[kThreads / 32], warp_pages[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Q = a.t.Q;
  uint32_t bad = 0;

  // Prefix sums in 64 bits (lengths are the caller's data), stored clamped: rows to
  // cap (without rows, cap 0, to INT32_MAX), pages to INT32_MAX, which no free stack reaches.
  const int64_t most_rows = a.t.cap > 0 ? a.t.cap : INT32_MAX;
  int64_t base_rows = 0, base_pages = 0;
  for (int i0 = 0; i0 < Q; i0 += kThreads) {
    const int i = i0 + tid;
    int64_t rows = 0, pages = 0;
    if (i < Q) {
      const int32_t c = length_of(a.t.ctx_len[i]), n = length_of(a.t.new_len[i]);
      const int32_t held = pages_of(c), all = pages_of(c + n);
      if (all > a.t.pt_stride && n > 0) bad |= kStatusBadBound;
      rows = n;
      pages = max(min(all, a.t.pt_stride) - held, 0);
    }
    int64_t sr = rows, sp = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t ur = __shfl_up_sync(0xffffffffu, sr, o), up = __shfl_up_sync(0xffffffffu, sp, o);
      if (lane >= o) {
        sr += ur;
        sp += up;
      }
    }
    if (lane == 31) {
      warp_rows[warp] = sr;
      warp_pages[warp] = sp;
    }
    __syncthreads();
    int64_t before_r = base_rows, before_p = base_pages;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        before_r += warp_rows[w];
        before_p += warp_pages[w];
      }
      base_rows += warp_rows[w];
      base_pages += warp_pages[w];
    }
    if (i < Q) {
      start[i] = static_cast<int32_t>(min(before_r + sr - rows, most_rows));
      taken[i] = static_cast<int32_t>(min(before_p + sp - pages, static_cast<int64_t>(INT32_MAX)));
    }
    __syncthreads();   // the warp sums are rewritten by the next chunk
  }
  if (tid == 0) {
    start[Q] = static_cast<int32_t>(min(base_rows, most_rows));
    taken[Q] = static_cast<int32_t>(min(base_pages, static_cast<int64_t>(INT32_MAX)));
    if (base_rows > most_rows) bad |= kStatusBadBound;
  }
  __syncthreads();
  const int32_t rows = start[Q], pages = taken[Q];
  const bool simple = a.t.mask == nullptr && a.t.parent == nullptr;
  const int32_t free_count = max(*a.t.free_count, 0);
  if (tid == 0 && pages > free_count) bad |= kStatusBadPage;
  if (blockIdx.x == 0 && tid == 0) *a.t.free_left = max(free_count - pages, 0);

  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = first; i <= Q; i += step) a.t.row_start[i] = start[i];

  // new table entries
  for (int64_t n = first; n < pages; n += step) {
    const int i = find_last(taken, Q, static_cast<int32_t>(n));
    const int32_t held = pages_of(length_of(a.t.ctx_len[i]));
    int32_t page = -1;
    if (n < free_count) {
      page = a.t.free_pages[free_count - 1 - n];
      if (page < 0 || page >= a.t.P) bad |= kStatusBadPage;
    }
    a.t.page_table[static_cast<int64_t>(i) * a.t.pt_stride + held + (n - taken[i])] = page;
  }

  // The first slot of request i's page pg, -1 without one.  ctx: the request's cached tokens.
  const auto base_of = [&](int i, int32_t ctx, int32_t pg) {
    int32_t page = -1;
    const int32_t held = pages_of(ctx);
    if (pg < a.t.pt_stride) {
      if (pg < held) {
        page = a.t.page_table[static_cast<int64_t>(i) * a.t.pt_stride + pg];
      } else {
        const int32_t n = taken[i] + (pg - held);
        if (n < free_count) page = a.t.free_pages[free_count - 1 - n];
      }
    }
    if (page >= 0 && page < a.t.P) return page * kPage;
    bad |= kStatusBadPage;
    return -1;
  };

  // rows: four consecutive ones per thread, a run of groups per CTA, so that a thread
  // looks its request up again only where the last one ended
  const int64_t run = static_cast<int64_t>(a.groups_per_cta) * kThreads * kRowsPerThread;
  const int64_t run_end = min((blockIdx.x + 1) * run, static_cast<int64_t>(a.t.cap));
  int i = 0;
  int32_t end = 0, ctx = 0, begin = 0;   // request i: its rows [begin, end), its cached tokens
  for (int64_t r0l = blockIdx.x * run + tid * kRowsPerThread; r0l < run_end; r0l += kThreads * kRowsPerThread) {
    const int32_t r0 = static_cast<int32_t>(r0l);
    int32_t req[kRowsPerThread], bound[kRowsPerThread], pos[kRowsPerThread], slot[kRowsPerThread];
    uint64_t mask[kRowsPerThread];
    if (r0 < rows && r0 >= end) {
      i = find_last(start, Q, r0);
      begin = start[i];
      end = start[i + 1];
      ctx = length_of(a.t.ctx_len[i]);
    }
    if (simple && r0 + kRowsPerThread <= min(rows, end)) {
      // all four in one request, no tree: consecutive positions on one page or two
      const int32_t at = ctx + (r0 - begin);
      const int32_t pg = static_cast<int32_t>(static_cast<uint32_t>(at) / kPage), tok = at % kPage;
      const int32_t base = base_of(i, ctx, pg);
      const int32_t next = tok + kRowsPerThread > kPage ? base_of(i, ctx, pg + 1) : -1;
#pragma unroll
      for (int k = 0; k < kRowsPerThread; ++k) {
        const bool here = tok + k < kPage;
        const int32_t b = here ? base : next;
        req[k] = i;
        bound[k] = at + k + 1;
        pos[k] = at + k;
        slot[k] = b < 0 ? -1 : b + (here ? tok + k : tok + k - kPage);
        mask[k] = 0;
      }
    } else {
      int32_t t = r0 < rows ? r0 - begin : 0, at = ctx + t, page_seen = -1, base = -1;
#pragma unroll
      for (int k = 0; k < kRowsPerThread; ++k, ++t, ++at) {
        const int32_t r = r0 + k;
        req[k] = 0;
        bound[k] = 0;
        pos[k] = 0;
        slot[k] = -1;
        mask[k] = 0;
        if (r >= rows) continue;
        if (r >= end) {   // the next request with rows
          do ++i;
          while (r >= start[i + 1]);
          t = 0;
          begin = r;
          end = start[i + 1];
          at = ctx = length_of(a.t.ctx_len[i]);
          page_seen = -1;
        }
        const int32_t pg = static_cast<int32_t>(static_cast<uint32_t>(at) / kPage);
        if (pg != page_seen) {
          page_seen = pg;
          base = base_of(i, at - t, pg);
        }
        // walk up the tree: parents are earlier tokens, so it ends within 64 steps
        int32_t depth = t;
        uint64_t m = 0;
        if (a.t.parent != nullptr && t < IDX_MAX_TREE) {
          depth = 0;
          int32_t u = t;
          for (;;) {
            m |= 1ull << u;
            const int32_t p = a.t.parent[start[i] + u];
            if (p < 0 || p >= u) {
              if (p != -1) bad |= kStatusBadBound;
              break;
            }
            u = p;
            ++depth;
          }
        } else if (t < IDX_MAX_TREE) {
          m = (2ull << t) - 1ull;   // bits 0 .. t (t = 63: the shift leaves 0, minus 1 sets all)
        }
        if (t >= IDX_MAX_TREE && (a.t.mask != nullptr || a.t.parent != nullptr)) bad |= kStatusBadBound;
        req[k] = i;
        bound[k] = at + 1;
        pos[k] = at - t + depth;
        slot[k] = base < 0 ? -1 : base + at % kPage;
        mask[k] = m;
      }
    }
    if (a.vec4 && r0 + kRowsPerThread <= a.t.cap) {
      *reinterpret_cast<int4 *>(a.t.row_req + r0) = make_int4(req[0], req[1], req[2], req[3]);
      *reinterpret_cast<int4 *>(a.t.row_bound + r0) = make_int4(bound[0], bound[1], bound[2], bound[3]);
      *reinterpret_cast<int4 *>(a.t.row_pos + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4 *>(a.t.slot + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.t.mask != nullptr) {
        reinterpret_cast<ulonglong2 *>(a.t.mask + r0)[0] = make_ulonglong2(mask[0], mask[1]);
        reinterpret_cast<ulonglong2 *>(a.t.mask + r0)[1] = make_ulonglong2(mask[2], mask[3]);
      }
    } else {
      for (int k = 0; k < kRowsPerThread && r0 + k < a.t.cap; ++k) {
        a.t.row_req[r0 + k] = req[k];
        a.t.row_bound[r0 + k] = bound[k];
        a.t.row_pos[r0 + k] = pos[k];
        a.t.slot[r0 + k] = slot[k];
        if (a.t.mask != nullptr) a.t.mask[r0 + k] = mask[k];
      }
    }
  }
  if (bad) flag_status(a.status, bad);
}

}  // namespace

cudaError_t launch_tree_tables(TreeTablesArgs a, int num_sms, cudaStream_t stream) {
  // enough CTAs for one row group per thread, at most about eight per SM (the sums
  // are repeated by every CTA)
  const int64_t groups = (static_cast<int64_t>(a.t.cap) + kThreads * kRowsPerThread - 1) / (kThreads * kRowsPerThread);
  const int64_t most = 8 * static_cast<int64_t>(num_sms);
  a.groups_per_cta = groups <= most ? 1 : static_cast<int32_t>((groups + most - 1) / most);
  const int64_t grid = groups < 1 ? 1 : (groups + a.groups_per_cta - 1) / a.groups_per_cta;
  const size_t smem = 2 * (static_cast<size_t>(a.t.Q) + 1) * sizeof(int32_t);
  tree_tables_kernel<<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace idx
