// ssdv_attn.cuh -- what the attention kernels over the 4-bit cache share:
// barriers, unpacking of codes, and the list of work.
//
// Work is split evenly whatever the lengths: every team (some warps, or a CTA)
// takes the same number of tiles of the list (request, kv head, pass over the
// rows, tile).  Rows whose tiles are split between teams leave partial sums in
// the workspace, slot 0 of a team for the part it begins with and slot 1 for one
// it begins later; a second kernel joins them in the teams' order, so results do
// not depend on timing.
#pragma once

#include "ssdv_kv.cuh"

#include <atomic>

// The attention kernels are compiled twice: without (0) and with (1) sinks, first
// positions and sums in place of outputs.  They are bound by instruction fetches and
// latency, and what those cost would be paid by all calls (64 requests of 201 to 8003
// tokens, 20 rows: 100 us without, 110 with; 2 of 131072: 172 and 210).
#ifndef SSDV_ATTN_MORE
#define SSDV_ATTN_MORE 0
#endif

namespace ssdv {

constexpr bool kMore = SSDV_ATTN_MORE;
constexpr int kBand = 29;        // octaves below that in which fp16 keeps 11 bits
constexpr int kBands = 5;        // passes a tile may take; weights below 2^-141 of its largest are dropped
constexpr float kSmallest = 6.103515625e-05f;  // 2^(kBias - kBand)
constexpr int kMaxSms = 160;     // the workspace is sized for this many CTAs

// How the rows of a kv head are spread: nt n-tiles per warp or pair, g groups of
// rows per team (all reading the same tile), rt passes over the cache; t teams
// per CTA with s stages each.
struct AttnShape {
  int nt, p, g, t, s, rt;
  bool tc;  // ssdv_attn_tc.cu: one team per CTA, nt n-tiles a pass
};

struct AttnLaunch {
  KvAttnArgs a;
  AttnShape p;
  int per;          // query heads per kv head
  int rows;         // nq * per
  int rows_pass;    // g * nt * 8
  int4* desc;       // [teams]: request, head * rt + pass, parts, first slot
  float2* ml;       // [2 teams, rows_pass]: maximum and sum of a part
  float* o;         // [2 teams, rows_pass, D]
};

cudaError_t launch_attention_tc(const AttnLaunch& L, int sms, cudaStream_t stream);
cudaError_t launch_attention_tc_more(const AttnLaunch& L, int sms, cudaStream_t stream);
cudaError_t launch_attention_more(const KvAttnArgs& a, int D, int esize, cudaStream_t stream);

#ifdef __CUDACC__

namespace {

// Lets a kernel use `bytes` of dynamic shared memory, once per device.
template <auto kKernel>
cudaError_t allow_shared(int bytes) {
  static std::atomic<unsigned long long> known{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (known.load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) known.fetch_or(1ull << dev);
  return e;
}

// Launches a kernel whose first act is to wait for the one before it (griddepcontrol.wait),
// so that its launch overlaps that one's end.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- mbarriers and bulk copies ----

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, int parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// True some 2^32 cycles (two seconds) after the first call with since = 0: every
// wait ends.
__device__ __forceinline__ bool late(long long& since) {
  const long long now = clock64();
  if (since == 0) since = now;
  return now - since > (1ll << 32);
}
// False if the phase did not complete within 2^24 tries of about a hundred cycles.
// The loop is as short as it gets: warps that wait take instruction fetches from
// those that work.
__device__ __forceinline__ bool bar_wait(uint32_t bar, int parity) {
#pragma unroll 1
  for (int i = 1 << 24; i; --i)
    if (bar_test(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, int bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// ---- unpacking ----

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// 16 + u of the pairs at bits 9:6, 256 + u of those at bits 5:2: one three-input
// operation each, for which the or-ed constants are kept in registers.
struct Bases {
  uint32_t hi, lo;
};
__device__ __forceinline__ Bases make_bases() {
  Bases b;
  asm volatile("mov.b32 %0, 0x4C004C00;\n\tmov.b32 %1, 0x5C005C00;" : "=r"(b.hi), "=r"(b.lo));
  return b;
}
__device__ __forceinline__ uint32_t pair_hi(uint32_t w, const Bases& b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x03C003C0, %2, 0xEA;" : "=r"(d) : "r"(w), "r"(b.hi));
  return d;
}
__device__ __forceinline__ uint32_t pair_lo(uint32_t w, const Bases& b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x003C003C, %2, 0xEA;" : "=r"(d) : "r"(w), "r"(b.lo));
  return d;
}
constexpr uint32_t kMinus24 = 0xCE00CE00u, kMinus264 = 0xDC20DC20u;  // fp16 pairs

__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t p, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t p, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t p, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(p), "r"(v.x), "r"(v.y) : "memory");
}

// ---- the list of work ----

// What a request's rows see together, and its tiles.
struct Span {
  int len, nq;     // query rows i < nq are real
  int lo, hi;      // positions some row sees, beside those below a.sinks
  // Tile t is tile0 + t of the sequence for t < ahead and t - ahead after that: the
  // tiles of sinks come last, so that their large scores do not become the
  // reference of a window's small ones.  At least one tile, so that some team
  // writes the outputs.
  int tile0, ahead, tiles;
  int first;
  bool bad, some;
  __device__ __forceinline__ int tile(int t) const { return !kMore || t < ahead ? tile0 + t : t - ahead; }
  __device__ __forceinline__ bool any() const { return kMore ? some : hi > lo; }  // some row sees something
};
__device__ __forceinline__ int sinks_of(const KvAttnArgs& a) { return kMore ? a.sinks : 0; }
__device__ __forceinline__ bool own_sums(const KvAttnArgs& a) { return kMore && a.own_ml; }
__device__ __forceinline__ int row_lo(const KvAttnArgs& a, const Span& s, int i) {
  return a.window ? max(0, s.len + i + 1 - a.window) : kMore ? s.first : 0;
}
template <int kTile>
__device__ __forceinline__ Span find_span(const KvAttnArgs& a, int b) {
  Span s;
  s.len = a.kv_len[b];
  s.nq = a.n_q ? a.n_q[b] : a.nq;
  s.bad = s.len < 0 || s.nq < 0 || s.nq > a.nq ||
          static_cast<long long>(s.len) + (a.past_only ? 0 : s.nq) >
              static_cast<long long>(a.c.max_pages) * a.c.page_size;
  s.lo = s.hi = s.tile0 = 0;
  s.tiles = 1;
  if (kMore) {
    s.first = 0;
    s.ahead = 1;
    s.some = false;
  }
  if (kMore && a.first) {
    s.first = a.first[b];
    s.bad |= s.first < 0 || s.first > s.len;
  }
  if (s.bad || s.nq == 0) return s;
  if constexpr (!kMore) {
    s.hi = a.past_only ? s.len : s.len + s.nq;
    s.lo = a.window ? max(0, s.len + 1 - a.window) : 0;
    if (s.lo >= s.hi) {
      s.lo = s.hi = 0;
      return s;
    }
    s.tile0 = s.lo / kTile;
    s.tiles = (s.hi + kTile - 1) / kTile - s.tile0;
    return s;
  }
  const int hi = a.past_only ? s.len : s.len + s.nq;
  const int lo = min(row_lo(a, s, 0), hi);
  const int sink_tiles = (min(sinks_of(a), lo) + kTile - 1) / kTile;
  const int tile0 = max(lo / kTile, sink_tiles), ahead = max((hi + kTile - 1) / kTile - tile0, 0);
  // (a window that lies behind the past holds nothing, whatever tile it ends in)
  const int seen = lo < hi ? ahead : 0;
  if (seen + sink_tiles == 0) return s;
  s.some = true;
  s.lo = lo;
  s.hi = hi;
  s.tile0 = tile0;
  s.ahead = seen;
  s.tiles = seen + sink_tiles;
  return s;
}
// Whether some row sees a position of a request.
__device__ __forceinline__ bool in_span(const KvAttnArgs& a, int lo, int hi, int pos) {
  return pos < hi && (pos >= lo || (kMore && pos < a.sinks));
}
__device__ __forceinline__ int row_hi(const KvAttnArgs& a, int len, int i) { return a.past_only ? len : len + i + 1; }

// A place in the list.
template <int kTile>
struct Place {
  int b, hr, tile;  // request, head * rt + pass, tile of the request's span
  Span s;
  __device__ __forceinline__ void next(const KvAttnArgs& a, int per_request) {
    if (++tile < s.tiles) return;
    tile = 0;
    if (++hr < per_request) return;
    hr = 0;
    if (++b < a.B) s = find_span<kTile>(a, b);
  }
};

// The CTA's view of the list: prefix sums of the requests' tiles.  Beginning and
// ending a row's tiles costs a team about as much as `extra` tiles, so that many
// units without work come before each row's tiles, and teams share units evenly.
template <int kTile>
struct List {
  const long long* scan;
  int chunk, threads, per_request, requests, extra;
  long long units, quota, tiles;
  struct Share {
    Place<kTile> at;   // its first tile
    int count;         // how many tiles
    int row_unit;      // unit where it begins, from that of the row's first tile
  };

  // The first tile at or after unit u < units, and how many come before it in the list.
  __device__ __forceinline__ Place<kTile> find(const KvAttnArgs& a, long long u, long long& rank, int& row_unit) const {
    const auto first = [&](int t) { return (scan[t] + static_cast<long long>(extra) * t * chunk) * per_request; };
    int lo = 0, hi = threads - 1;  // last thread whose requests begin at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (mid * chunk < requests && first(mid) <= u) lo = mid;
      else hi = mid - 1;
    }
    Place<kTile> at;
    at.b = lo * chunk;
    long long u0 = first(lo);
    rank = scan[lo] * per_request;
    at.s = find_span<kTile>(a, at.b);
    for (;;) {
      const long long mine = static_cast<long long>(at.s.tiles) * per_request;
      if (u0 + mine + static_cast<long long>(extra) * per_request > u) break;
      u0 += mine + static_cast<long long>(extra) * per_request;
      rank += mine;
      at.s = find_span<kTile>(a, ++at.b);
    }
    const long long k = u - u0;
    at.hr = static_cast<int>(k / (at.s.tiles + extra));
    row_unit = static_cast<int>(k % (at.s.tiles + extra)) - extra;
    at.tile = max(row_unit, 0);
    rank += static_cast<long long>(at.hr) * at.s.tiles + at.tile;
    return at;
  }
  // A team's tiles.
  __device__ __forceinline__ Share share(const KvAttnArgs& a, long long me) const {
    Share x = {};
    const long long begin = me * quota;
    if (begin >= units) return x;
    long long rank, end = tiles;
    int unused;
    x.at = find(a, begin, rank, x.row_unit);
    if (extra == 0) end = min(units, begin + quota);
    else if (begin + quota < units) find(a, begin + quota, end, unused);
    x.count = static_cast<int>(end - rank);
    return x;
  }

  // All threads of the CTA; ends with a barrier.  `sums` holds a number per warp.
  __device__ __forceinline__ void build(const KvAttnArgs& a, int heads_passes, int teams, int extra_, long long* scan_,
                                        long long* sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    scan = scan_;
    threads = blockDim.x;
    chunk = (a.B + threads - 1) / threads;
    per_request = heads_passes;
    requests = a.B;
    long long mine = 0;
#pragma unroll 1
    for (int b = tid * chunk; b < min(a.B, (tid + 1) * chunk); ++b) mine += find_span<kTile>(a, b).tiles;
    long long x = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll 1
    for (int v = 0; v < threads / 32; ++v) {
      if (v < warp) before += sums[v];
      total += sums[v];
    }
    scan_[tid] = before + x - mine;
    __syncthreads();
    tiles = total * per_request;
    // (with few tiles a team, whole tiles count for more than the beginnings do)
    extra = static_cast<int>(min(static_cast<long long>(extra_), tiles / teams / 2));
    units = tiles + static_cast<long long>(extra) * requests * per_request;
    quota = (units + teams - 1) / teams;
  }
  // What a team that begins a row of `tiles` tiles, the first at unit seg, says of its parts.
  __device__ __forceinline__ int2 row_parts(long long seg, int tiles, long long me) const {
    return make_int2(static_cast<int>((seg + tiles - 1) / quota - me + 1),
                     static_cast<int>(2 * me + (seg - extra > me * quota ? 1 : 0)));
  }
  // What a team writes about the parts it begins with: the first team to begin
  // inside a row's tiles, past the first of them, has that row's parts joined.
  __device__ __forceinline__ int4 parts(const Share& x, long long me) const {
    if (x.count == 0) return make_int4(0, 0, 0, 0);
    const long long seg = me * quota - x.row_unit, prev = seg / quota;
    int4 d = make_int4(x.at.b, x.at.hr, 0, 0);
    if (x.at.tile > 0 && prev == me - 1) {
      d.z = static_cast<int>((seg + x.at.s.tiles - 1) / quota - prev + 1);
      d.w = static_cast<int>(2 * prev + (seg - extra > prev * quota ? 1 : 0));
    }
    return d;
  }
};

}  // namespace

#endif  // __CUDACC__

}  // namespace ssdv
