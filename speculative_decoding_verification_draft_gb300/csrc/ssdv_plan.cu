// ssdv_plan.cu -- page tables, held pages and slots from the requests' lengths.
//
// Request b is to hold h_b = max(shared_b, ceil((len_b + new_b) / page_size))
// pages.  What it holds beyond that goes onto the stack of free pages, in the
// order of requests and columns; then what requests lack is taken from the
// stack's top in the same order, from all that want pages while the running sum
// of wants stays within the stack.  With G_b and W_b the sums of pages given and
// wanted by the requests before b, the k-th page that b gives lands at place
// n_free + G_b + k, and the k-th that it takes lies at n_free + G - 1 - W_b - k: two
// prefix sums over the batch, and every page has its place.
//
// Where no output is an input, one kernel of many CTAs does it all, each CTA going through
// the sums again.  In place, one CTA does the sums and moves pages; the rest, copies and
// slots, is spread over the GPU by a second kernel when it is large.
//
// Measured: 64 requests of a round, two ended and two beginning with up to 1500 tokens: 8
// us (in place 10); 512 requests, 61 ended and 97 beginning: 13 us for 9.7 MB (in place
// 18).  Chains of dependent loads take most: lengths, sums, pages, the stack.  In a
// program the calls take 24 and 28 us each, which is the host's time.
#include "ssdv_round.cuh"

#include <algorithm>

#include "ssdv.h"

namespace ssdv {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kChunk = 256;  // cells of a row, or slots, that a warp takes at a time
// In place: cells (of the table, the stack and the slots) up to which the one CTA also
// copies and writes slots; above, a second kernel does, four CTAs an SM.  One against two:
// 6.4 and 7.8 us for 1,000 cells, 8.0 and 11.1 for 5,000, 11.9 and 9.3 for 24,000, 22.6
// and 10.2 for 110,000.
constexpr long long kAlone = 16384;
// Not in place: one kernel of many CTAs (4.6, 8.4, 8.1 and 8.0 us for these), as long as
// the plan of a batch fits 48 KB of shared memory.
constexpr int kAllThreads = 512, kAllRequests = 2048;

struct Want {
  int held, hold;
  bool bad;
};
__device__ __forceinline__ Want look(const KvPlanArgs& a, int b) {
  Want w;
  const int len = a.len[b], add = a.n_new ? a.n_new[b] : a.n, shared = a.shared ? a.shared[b] : 0;
  w.held = a.held[b];
  const long long end = static_cast<long long>(len) + add;
  w.bad = len < 0 || add < 0 || add > a.n || end > static_cast<long long>(a.max_pages) * a.page_size || w.held < 0 ||
          w.held > a.max_pages || shared < 0 || shared > w.held;
  w.hold = w.bad ? w.held : max(shared, static_cast<int>((end + a.page_size - 1) / a.page_size));
  return w;
}

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// Inclusive sum over the CTA's kWarps warps; total gets the sum of all.
template <int kWarps>
__device__ __forceinline__ long long block_scan(long long x, long long* sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_scan(x, lane);
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  const long long s = warp_scan(lane < kWarps ? sums[lane] : 0, lane);
  total = __shfl_sync(~0u, s, 31);
  const long long before = __shfl_sync(~0u, s, max(warp - 1, 0));
  return x + (warp ? before : 0);
}

// What is left once pages have moved: cells that did not change, the stack's
// rest, and the slots, by `warps` warps.
__device__ __forceinline__ void finish(const KvPlanArgs& a, long long me, long long warps, int lane) {
  const int4 head = a.work[0];  // free pages before, on the stack at its highest, after
  const int4* plan = a.work + 1;
  if (a.out_free != a.free) {
    const int keep = min(head.x, head.z);
    for (long long i = me * 32 + lane; i < a.n_pages; i += warps * 32)
      if (i < keep || i >= head.y) a.out_free[i] = a.free[i];
  }
  if (a.out_table != a.table) {
    const int per = (a.max_pages + kChunk - 1) / kChunk;
    for (long long u = me; u < static_cast<long long>(a.B) * per; u += warps) {
      const int b = static_cast<int>(u / per), c0 = static_cast<int>(u % per) * kChunk;
      const int4 p = plan[b];
      const long long row = static_cast<long long>(b) * a.max_pages;
      const int lo = min(p.x, p.y), hi = max(p.x, p.y), end = min(c0 + kChunk, a.max_pages);
#pragma unroll 4
      for (int c = c0 + lane; c < end; c += 32)
        if (c < lo || c >= hi) a.out_table[row + c] = a.table[row + c];
    }
  }
  if (a.slots) {
    const int per = (a.n + kChunk - 1) / kChunk;
    for (long long u = me; u < static_cast<long long>(a.B) * per; u += warps) {
      const int b = static_cast<int>(u / per), i0 = static_cast<int>(u % per) * kChunk;
      const int4 p = plan[b];
      const long long row = static_cast<long long>(b) * a.max_pages;
      const int len = a.len[b], add = p.w ? (a.n_new ? a.n_new[b] : a.n) : 0, end = min(i0 + kChunk, a.n);
      int64_t* out = a.slots + static_cast<long long>(b) * a.n;
#pragma unroll 4
      for (int i = i0 + lane; i < end; i += 32) {
        long long slot = -1;
        if (i < add) {
          const unsigned pos = len + i, col = pos / static_cast<unsigned>(a.page_size);
          // columns taken in this call are in the new table already
          const int page = (col >= static_cast<unsigned>(p.x) ? a.out_table : a.table)[row + col];
          if (page >= 0) slot = static_cast<long long>(page) * a.page_size + (pos - col * a.page_size);
        }
        out[i] = slot;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const __grid_constant__ KvPlanArgs a, bool alone) {
  __shared__ long long sums[kWarps];
  __shared__ unsigned long long taken;
  __shared__ int errors;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    taken = 0;
    errors = 0;
  }
  const int n_free = a.n_free[0];
  // pages given back by all
  long long given = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    long long mine = 0, sum;
    if (b0 + tid < a.B) {
      const Want w = look(a, b0 + tid);
      mine = max(w.held - w.hold, 0);
    }
    block_scan<kWarps>(mine, sums, sum);
    given += sum;
  }
  const long long total = n_free + given;
  const bool broken = n_free < 0 || n_free > a.n_pages || total > a.n_pages;
  // each request's place among those that give and those that take
  int4* plan = a.work + 1;
  long long gives = 0, wants = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    Want w = {0, 0, false};
    if (b < a.B) w = look(a, b);
    const int give = max(w.held - w.hold, 0), want = max(w.hold - w.held, 0);
    long long sum_gives, sum_wants;
    const long long g = gives + block_scan<kWarps>(give, sums, sum_gives), t = wants + block_scan<kWarps>(want, sums, sum_wants);
    gives += sum_gives;
    wants += sum_wants;
    if (b < a.B) {
      const bool served = !w.bad && !broken && (want == 0 || t <= total);
      const int after = served ? w.hold : w.held;
      plan[b] = w.bad ? make_int4(0, 0, 0, 0)
                      : make_int4(w.held, after, static_cast<int>(give ? g - give : t - want), served);
      a.out_held[b] = after;
      if (served && want) atomicMax(&taken, static_cast<unsigned long long>(t));
      if (w.bad) atomicOr(&errors, 1 << SSD_ERR_LENGTH);
      else if (!served && !broken) atomicOr(&errors, 1 << SSD_ERR_POOL);
    }
  }
  __syncthreads();
  const int left = broken ? n_free : static_cast<int>(total - static_cast<long long>(taken));
  if (tid == 0) {
    a.out_n_free[0] = left;
    // (a broken stack is copied as it is)
    a.work[0] = broken ? make_int4(0, 0, 0, 0) : make_int4(n_free, static_cast<int>(total), left, 0);
    if (broken) atomicOr(&errors, 1 << SSD_ERR_PAGE);
    if (errors) atomicOr(a.status, errors);
  }
  // pages that come back, then pages that go: a warp looks at 32 requests at a time
  const int top = static_cast<int>(total) - 1;
  for (int pass = 0; pass < 2; ++pass) {
    for (int b0 = warp * 32; b0 < a.B; b0 += kThreads) {
      const int4 p = b0 + lane < a.B ? plan[b0 + lane] : make_int4(0, 0, 0, 0);
      unsigned todo = __ballot_sync(~0u, pass == 0 ? p.y < p.x : p.y > p.x);
      while (todo) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const int held = __shfl_sync(~0u, p.x, l), after = __shfl_sync(~0u, p.y, l), rank = __shfl_sync(~0u, p.z, l);
        const long long row = static_cast<long long>(b0 + l) * a.max_pages;
        // (four loads a lane before the first store: the arrays may be the same)
        for (int c0 = min(held, after) + lane; c0 < max(held, after); c0 += 128) {
          int page[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int c = c0 + 32 * x;
            if (pass == 0) {
              if (c < held) page[x] = a.table[row + c];
            } else if (c < after) {
              const int at = top - (rank + c - held);
              page[x] = at >= n_free ? a.out_free[at] : a.free[at];
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int c = c0 + 32 * x;
            if (pass == 0) {
              if (c < held) {
                a.out_free[n_free + rank + c - after] = page[x];
                a.out_table[row + c] = -1;
              }
            } else if (c < after) {
              a.out_table[row + c] = page[x];
              a.out_free[top - (rank + c - held)] = -1;
            }
          }
        }
      }
    }
    __syncthreads();
  }
  if (alone) finish(a, warp, kWarps, lane);
}

__global__ void __launch_bounds__(256) kv_plan_finish_kernel(const __grid_constant__ KvPlanArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  finish(a, static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5), static_cast<long long>(gridDim.x) * 8,
         threadIdx.x & 31);
}

// The same in one kernel, where no output is an input: every CTA goes through the sums
// and writes its share of the outputs from the inputs alone.  A place of the stack at or
// above n_free is a page that is given back, found by its rank among those.
__global__ void __launch_bounds__(kAllThreads) kv_plan_all_kernel(const __grid_constant__ KvPlanArgs a) {
  extern __shared__ int4 plan[];  // [B]: held, after, first rank of what it takes, served; then the pages given before it
  __shared__ long long sums[kAllThreads / 32];
  __shared__ unsigned long long taken_, errors_;
  int* given_before = reinterpret_cast<int*>(plan + a.B);
  constexpr int W = kAllThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) taken_ = errors_ = 0;
  const int n_free = a.n_free[0];
  long long given = 0, wants = 0;
  for (int b0 = 0; b0 < a.B; b0 += kAllThreads) {
    const int b = b0 + tid;
    Want w = {0, 0, false};
    if (b < a.B) w = look(a, b);
    const int give = max(w.held - w.hold, 0), want = max(w.hold - w.held, 0);
    long long sum_gives, sum_wants;
    const long long g = given + block_scan<W>(give, sums, sum_gives), t = wants + block_scan<W>(want, sums, sum_wants);
    given += sum_gives;
    wants += sum_wants;
    if (b < a.B) {
      // (sums beyond the stack are cut: such a request is not served)
      plan[b] = make_int4(w.held, w.hold, static_cast<int>(min(t - want, 0x7FFFFFFFll)), w.bad ? -1 : 0);
      given_before[b] = static_cast<int>(min(g - give, 0x7FFFFFFFll));
    }
  }
  __syncthreads();
  const long long total = n_free + given;
  const bool broken = n_free < 0 || n_free > a.n_pages || total > a.n_pages;
  for (int b = tid; b < a.B; b += kAllThreads) {
    int4 p = plan[b];
    const bool bad = p.w < 0;
    const long long end = static_cast<long long>(p.z) + (p.y - p.x);  // of what it takes
    const bool served = !bad && !broken && (p.y <= p.x || end <= total);
    if (served && p.y > p.x) atomicMax(&taken_, static_cast<unsigned long long>(end));
    if (bad || !served) atomicOr(&errors_, bad ? 1ull << SSD_ERR_LENGTH : broken ? 0ull : 1ull << SSD_ERR_POOL);
    p.w = served;
    if (!served) p.y = p.x;
    plan[b] = p;
    if (blockIdx.x == 0) a.out_held[b] = p.y;
  }
  __syncthreads();
  const int left = broken ? n_free : static_cast<int>(total - static_cast<long long>(taken_));
  const int top = static_cast<int>(total) - 1;
  if (blockIdx.x == 0 && tid == 0) {
    a.out_n_free[0] = left;
    const int errors = static_cast<int>(errors_) | (broken ? 1 << SSD_ERR_PAGE : 0);
    if (errors) atomicOr(a.status, errors);
  }
  const auto on_stack = [&](int at) {  // place `at` once all that is given back lies there
    if (at < n_free) return a.free[at];
    const int r = at - n_free;
    int lo = 0, hi = a.B - 1;  // the last request with no more than r pages given before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (given_before[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    return a.table[static_cast<long long>(lo) * a.max_pages + plan[lo].y + r - given_before[lo]];
  };
  const long long me = static_cast<long long>(blockIdx.x) * W + (tid >> 5), warps = static_cast<long long>(gridDim.x) * W;
  for (long long i = me * 32 + lane; i < a.n_pages; i += warps * 32)
    a.out_free[i] = broken || i >= total ? a.free[i] : i < left ? on_stack(static_cast<int>(i)) : -1;
  const int per = (a.max_pages + kChunk - 1) / kChunk;
  for (long long u = me; u < static_cast<long long>(a.B) * per; u += warps) {
    const int b = static_cast<int>(u / per), c0 = static_cast<int>(u % per) * kChunk;
    const int4 p = plan[b];
    const long long row = static_cast<long long>(b) * a.max_pages;
    const int end = min(c0 + kChunk, a.max_pages);
#pragma unroll 4
    for (int c = c0 + lane; c < end; c += 32) {
      int page;
      if (c < min(p.x, p.y) || c >= max(p.x, p.y)) page = a.table[row + c];
      else page = p.y < p.x ? -1 : on_stack(top - (p.z + c - p.x));
      a.out_table[row + c] = page;
    }
  }
  if (!a.slots) return;
  const int chunks = (a.n + kChunk - 1) / kChunk;
  for (long long u = me; u < static_cast<long long>(a.B) * chunks; u += warps) {
    const int b = static_cast<int>(u / chunks), i0 = static_cast<int>(u % chunks) * kChunk;
    const int4 p = plan[b];
    const long long row = static_cast<long long>(b) * a.max_pages;
    const int len = a.len[b], add = p.w ? (a.n_new ? a.n_new[b] : a.n) : 0, end = min(i0 + kChunk, a.n);
    int64_t* out = a.slots + static_cast<long long>(b) * a.n;
#pragma unroll 4
    for (int i = i0 + lane; i < end; i += 32) {
      long long slot = -1;
      if (i < add) {
        const unsigned pos = len + i, col = pos / static_cast<unsigned>(a.page_size);
        const int c = static_cast<int>(col);
        const int page = c < p.x ? a.table[row + c] : on_stack(top - (p.z + c - p.x));
        if (page >= 0) slot = static_cast<long long>(page) * a.page_size + (pos - col * a.page_size);
      }
      out[i] = slot;
    }
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  long long cells = a.slots ? static_cast<long long>(a.B) * a.n : 0;
  if (a.out_table != a.table) cells += static_cast<long long>(a.B) * a.max_pages;
  if (a.out_free != a.free) cells += a.n_pages;
  const bool alone = cells <= kAlone;
  const auto blocks = [&](long long per) { return static_cast<unsigned>(std::min((cells + per - 1) / per, 608ll)); };
  if (a.B <= kAllRequests && a.out_table != a.table && a.out_held != a.held && a.out_free != a.free &&
      a.out_n_free != a.n_free) {
    const unsigned grid = std::min(blocks(kAllThreads / 32 * kChunk), 304u);
    kv_plan_all_kernel<<<grid, kAllThreads, a.B * (sizeof(int4) + 4), stream>>>(a);
    return cudaGetLastError();
  }
  kv_plan_kernel<<<1, kThreads, 0, stream>>>(a, alone);
  cudaError_t e = cudaGetLastError();
  if (alone || e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks(8 * kChunk));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_plan_finish_kernel, a);
}

}  // namespace ssdv
