// Step plan: block tables, slot maps and positions from request lengths.
//
// With c_b cached and n_b new tokens and pages of p tokens, request b opens
// take_b = ceil((c_b + n_b)/p) - ceil(c_b/p) pages.  Exclusive sums over the
// requests of n_b and take_b number the step's tokens and its new pages; token
// t of request b is at position c_b + t, on the page that the block table
// already has (position below ceil(c_b/p)*p) or on the new page of that index,
// which every block reads from the free list itself, so that no block waits
// for another one's table writes.
//
// Every block forms the sums of all requests (1024 at a time in shared
// memory: a few bytes per request, read through L2) and takes every G-th tile
// of 256 tokens and of 256 pages: one launch, no communication between blocks.
// A decode batch is one or two blocks and its time is launch plus four
// dependent round trips (lengths, sums, page, store); the bytes of a step
// (16 per token) never bound it.  A call takes 6.6 us for 256 decode requests and
// 7.4 us for 129 requests with 64K new tokens, most of it on the host (replayed in
// a graph 3.9 and 4.7; 3.6 and 195 where the lengths advance in place).
#include "common.cuh"
#include "launch.h"
#include "serving.h"

namespace idx {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;
constexpr int kChunk = kThreads * kPerThread;

struct ChunkReq {
  int32_t cached;
  int32_t have;  // pages it has
};

// Last b in [0, n) with start[b] <= x (start[0] <= x).
__device__ __forceinline__ int last_at_or_below(const long long* start, int n, long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_step_kernel(PlanArgs a) {
  __shared__ long long tok_start[kChunk + 1];
  __shared__ long long page_start[kChunk + 1];
  __shared__ ChunkReq req[kChunk];
  __shared__ long long warp_tok[kThreads / 32], warp_page[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << a.page_shift;
  pdl_launch_dependents();
  pdl_wait();  // inputs may come from the previous kernel
  int head = *a.head;
  head = head < 0 || head > a.num_free ? a.num_free : head;
  long long tok_base = 0, page_base = 0;
  int bad = 0;  // counted by this thread

  // page id at entry x of the free list (x counted from the head), or -1
  auto free_page = [&](long long x) -> int {
    if (x >= a.num_free - head) return -1;
    const int id = __ldg(a.free_pages + head + x);
    return id < 0 || id >= a.num_blocks ? -1 : id;
  };

  for (int b0 = 0, chunk = 0; b0 < a.B; b0 += kChunk, ++chunk) {
    const int nb = min(kChunk, a.B - b0);
    const bool mine = chunk % (int)gridDim.x == (int)blockIdx.x;
    long long tok[kPerThread], pages[kPerThread], st = 0, sp = 0;
    int lens[kPerThread], adds[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int r = tid * kPerThread + i;
      // not through the read-only path: context_lens may be this array
      lens[i] = r < nb ? a.cached[b0 + r] : 0;
      adds[i] = r < nb ? __ldg(a.fresh + b0 + r) : 0;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int r = tid * kPerThread + i;
      int cached = lens[i], fresh = adds[i];
      if (r < nb) {
        if (cached < 0 || fresh < 0) {
          if (mine) ++bad;
          cached = fresh = 0;
        }
        if ((long long)cached + fresh > INT32_MAX) {
          if (mine) ++bad;
          fresh = 0;
        }
      }
      const long long ctx = (long long)cached + fresh;
      const long long want = (ctx + page - 1) >> a.page_shift;
      const long long have = ((long long)cached + page - 1) >> a.page_shift;
      if (mine && r < nb) {
        a.context_lens[b0 + r] = (int32_t)ctx;
        if (want > a.max_blocks) ++bad;
      }
      tok[i] = fresh;
      pages[i] = max(0ll, min(want, (long long)a.max_blocks) - have);
      if (r < kChunk) req[r] = ChunkReq{cached, (int32_t)have};
      st += tok[i];
      sp += pages[i];
    }
    long long xt = st, xp = sp;  // inclusive sums over the warp, then the block
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long yt = __shfl_up_sync(~0u, xt, d), yp = __shfl_up_sync(~0u, xp, d);
      if (lane >= d) {
        xt += yt;
        xp += yp;
      }
    }
    if (lane == 31) {
      warp_tok[warp] = xt;
      warp_page[warp] = xp;
    }
    __syncthreads();
    xt -= st;
    xp -= sp;
    for (int w = 0; w < warp; ++w) {
      xt += warp_tok[w];
      xp += warp_page[w];
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int r = tid * kPerThread + i;
      tok_start[r] = xt;
      page_start[r] = xp;
      if (mine && r < nb)
        a.query_start[b0 + r] = (int32_t)min(tok_base + xt, (long long)INT32_MAX);
      xt += tok[i];
      xp += pages[i];
    }
    if (tid == kThreads - 1) {
      tok_start[kChunk] = xt;
      page_start[kChunk] = xp;
    }
    __syncthreads();
    const long long ntok = tok_start[kChunk], npage = page_start[kChunk];

    // new pages of this chunk's requests
    for (long long x = (long long)blockIdx.x * kThreads + tid; x < npage;
         x += (long long)gridDim.x * kThreads) {
      const int r = last_at_or_below(page_start, kChunk, x);
      const int id = free_page(page_base + x);
      if (id < 0) ++bad;
      a.block_table[(int64_t)(b0 + r) * a.max_blocks + req[r].have + (x - page_start[r])] = id;
    }
    // its tokens
    for (long long x = (long long)blockIdx.x * kThreads + tid; x < ntok;
         x += (long long)gridDim.x * kThreads) {
      const long long t = tok_base + x;
      if (t >= a.num_tokens) break;
      const int r = last_at_or_below(tok_start, kChunk, x);
      const int pos = req[r].cached + (int)(x - tok_start[r]);
      const int pg = pos >> a.page_shift;
      int id = -1;
      if (pg >= req[r].have) {
        if (pg < a.max_blocks) id = free_page(page_base + page_start[r] + (pg - req[r].have));
      } else if (pg < a.max_blocks) {
        id = a.block_table[(int64_t)(b0 + r) * a.max_blocks + pg];
        if (id < 0 || id >= a.num_blocks) {
          id = -1;
          ++bad;
        }
      }
      a.slots[t] = id < 0 ? -1 : ((int64_t)id << a.page_shift) + (pos & (page - 1));
      a.positions[t] = pos;
      a.token_seq[t] = b0 + r;
    }
    tok_base += ntok;
    page_base += npage;
    __syncthreads();  // the shared sums are overwritten by the next chunk
  }

  for (long long t = tok_base + (long long)blockIdx.x * kThreads + tid; t < a.num_tokens;
       t += (long long)gridDim.x * kThreads) {
    a.slots[t] = -1;
    a.positions[t] = 0;
    a.token_seq[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.query_start[a.B] = (int32_t)min(tok_base, (long long)INT32_MAX);
    *a.head_out = (int32_t)min((long long)head + page_base, (long long)a.num_free);
    const long long over = tok_base - a.num_tokens;
    if (over > 0) bad += (int)min(over, 1ll << 30);
  }
  count_bad_input(a.errors, bad);
}

}  // namespace

cudaError_t launch_plan_step(const PlanArgs& a, int sms, cudaStream_t stream) {
  // One block per 256 tokens (a request's pages follow its tokens), at most one per
  // SM.  Where the lengths are advanced in place, one block in all: every block sums
  // all lengths, and here they change as it goes (each by the thread that has read it).
  const int64_t want = a.context_lens == a.cached ? 1 : (a.num_tokens + kThreads - 1) / kThreads;
  const int grid = (int)(want < 1 ? 1 : (want > sms ? sms : want));
  return launch_dependent(plan_step_kernel, dim3(grid), dim3(kThreads), 0, stream, a);
}

}  // namespace idx
