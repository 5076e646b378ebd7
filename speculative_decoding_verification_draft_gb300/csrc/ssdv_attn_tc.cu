// ssdv_attn_tc.cu -- attention over the 4-bit cache on the fifth-generation
// tensor cores (tcgen05, accumulators and unpacked codes in tensor memory):
// bf16 queries, 128 elements a head.
//
// The mathematics is that of ssdv_attn.cu, on tiles of 128 tokens, one CTA per
// SM, each taking an even share of the list of tiles:
//   S^T [128 tokens x N rows]    = K Q^T       M = 128 tokens, contraction 128 elements
//   O^T [128 elements x N rows] += V^T P^T     M = 128 elements, contraction 128 tokens
// The cache's side is the M side of both products, so rows (query tokens x query
// heads of a kv head) cost 16 at a time, and it goes from its codes through
// registers straight into tensor memory: a key row belongs to one lane, an
// element of the values to one lane, and only queries and weights, which are
// small, are operands in shared memory.  (Operands of 128 x 128 fp16 through
// shared memory would cost 512 of its cycles a tile for each product, more than
// the tile's share of the DRAM bandwidth allows.)
//
// Twenty warps with one job each, joined by mbarriers:
//   0-7   weights: scores from tensor memory, softmax, weights to shared memory
//         (warps 0-3 the first half of the rows, 4-7 the second)
//   8-11  keys: codes to tensor memory
//   12-15 values: codes to tensor memory; corrections of the sums; results
//   16    finds the CTA's parts of the list, bulk copies of the tiles' blocks
//   17    issues the scores' matrix instructions   18  the sums'   19  queries
// Every buffer is double, so that a tile's scores, the tile before's weights and
// the values of both overlap.
//
// Weights are fp16, 2^(x - m + kFast), with m a maximum of the row so far; while
// all of a tile's lie in [2^-14, 2^15], where fp16 keeps 11 bits, its products are
// added up in tensor memory and m stays.  Otherwise m follows the row's maximum,
// the values' warps rescale the sums, and weights below 2^-14 are passed over
// again, kBand octaves a pass, into a sum of their own that is added with its
// power of two.  Sums of weights and maxima are fp32.
//
// Measured: 256 requests of 2048 tokens, 40 rows: 388 us, 1.6 TB/s and 221 TFLOP/s
// of the products that count, a tile of 128 tokens in 1.8 us a CTA where the matrix
// instructions alone would take 0.55 (16 of 64 cycles each).  Nothing is saturated:
// about 1500 instructions a scheduler and tile issue at 0.5 a cycle, a tile passes
// four handshakes and two tiles overlap, and five roles fetch from one instruction
// cache, so loops are kept short and slow paths rolled up.  Tiles that are passed
// over again cost most: 64 requests of 201 to 8003 tokens, 20 rows, take 101 us, 301
// with scores spread four times as far, 265 with a first token that draws most of
// the weight.
#include "ssdv_attn.cuh"
#include "ssdv_tc.cuh"

#include <algorithm>

namespace ssdv {

namespace {

constexpr int kTile = 128;
constexpr int kBlocks = kTile / kKvBlock;
constexpr int kD = 128;
constexpr int kThreads = 640;
constexpr int kFast = 9, kTop = 15;
constexpr int kMaxStages = 8;
constexpr float kBandUp = 536870912.f;  // 2^kBand
// Beginning and ending a row's tiles costs as much as this many (64 requests of 97 to
// 4099 tokens, 40 rows: 201 us at 0 and 138 at 2 in an earlier form; now 90 at 3, 85
// at 4, 86 at 5, and 512 requests of up to 36 rows 96, 94 and 97).
constexpr int kPartTiles = 4;
constexpr int kRing = 8;  // parts described ahead
// Blocks lie 16 bytes past a multiple of 128 apart: the eight lanes of a phase,
// four blocks' two tokens, then read different banks.
constexpr int kBlockStride = kv_block_bytes(kD) + 16;
constexpr int kStage = kBlocks * kBlockStride;
constexpr int kHead = 1024;
constexpr int kSmem = 226000;

// Barriers, 8 bytes each from the start of shared memory.
enum : int {
  kFull = 0,            // [stages] a tile's bytes have arrived
  kEmpty = 8,           // [stages] keys and values have read them
  kKeysFull = 16,       // [2] keys unpacked            -> matrix
  kKeysEmpty = 18,      // [2] scores computed          -> keys
  kScoresFull = 20,     // [2] scores computed          -> weights
  kScoresEmpty = 22,    // [2] scores read              -> matrix
  kWeightsFull = 24,    // [2] weights written          -> matrix
  kWeightsEmpty = 26,   // [2] product computed         -> weights
  kValuesFull = 28,     // [2] values unpacked          -> matrix
  kValuesEmpty = 30,    // [2] tile's products computed -> values
  kOutFull = 32,        // [2] a part's products are all added -> values
  kOutEmpty = 34,       // [2] its sums read            -> matrix
  kInfoEmpty = 36,      // [2] a tile's word read       -> weights
  kQueryFull = 38,      // [2] queries written          -> matrix, weights
  kQueryEmpty = 40,     // [2] queries done with        -> queries
  kEndFull = 42,        // a part's sums and maxima     -> values
  kEndEmpty = 43,       // read                         -> weights
  kFixFull = 44,        // products so far added, or a band's computed -> values
  kFixDone = 45,        // sums corrected               -> matrix
  kDone = 46,           // all matrix instructions are done
  kPartFull = 48,       // [kRing] a part is described      -> all
  kPartEmpty = 56,      // [kRing] all have done with it    -> plan
  kBars = 64
};

// Shared memory after the head, for N rows.
template <int N>
struct Smem {
  static constexpr int kQueries = N * 256;      // N rows x 128 fp16, in 128-byte swizzled halves
  static constexpr int kWeights = kTile * 128;  // 128 tokens x 64 fp16, 128-byte swizzled
  static constexpr int query = kHead;
  static constexpr int weight = query + 2 * kQueries;
  static constexpr int table = weight + 2 * kWeights;   // [2] the values' scales and offsets: 8 pairs x 8 blocks x 8 groups
  static constexpr int nans = table + 2 * 4096;         // [2][8 blocks][8 groups][2] bytes
  static constexpr int fr = nans + 2 * 128;             // [N / 2] two rows' factors, then references
  static constexpr int maxima = fr + 8 * N;             // [N]
  static constexpr int tops = maxima + 4 * N;           // [4][N]
  static constexpr int fall = tops + 16 * N;            // [2][N]
  static constexpr int factors = fall + 8 * N;          // [2][N]
  static constexpr int ends = factors + 8 * N;          // [4][N] sums, [N] maxima
  static constexpr int rows = ends + 20 * N;            // [N] a finished row's factor, then which are zero
  static constexpr int results = (rows + 4 * N + 8 + 15) / 16 * 16;  // [N][128] bf16
  static constexpr int parts = results + 256 * N;       // [kRing] 64 bytes
  static constexpr int words = parts + 64 * kRing;           // info [2], bands, tensor memory address, flags [8]
  static constexpr int stages = (words + 64 + 127) / 128 * 128;
  static constexpr int kStages = (kSmem - stages) / kStage < kMaxStages ? (kSmem - stages) / kStage : kMaxStages;
  static constexpr int total = stages + kStages * kStage + 1024;  // the operands begin at a multiple of 1024
};
constexpr int kInfoRescale = 1, kInfoLast = 2;  // and the band from bit 8

// Tensor memory columns: keys and values twice 64 (128 fp16 a lane), scores twice
// N, sums of a part once or twice N, a band's products N.
template <int N>
struct Tmem {
  static constexpr int kOuts = N <= 48 ? 2 : 1;
  static constexpr int keys = 0, values = 128, scores = 256, outs = 256 + 2 * N, band = outs + kOuts * N;
  static_assert(band + N <= 512, "tensor memory");
};

// A CTA's share of the list, part by part: tiles of one (request, head, pass).
// One warp finds them (64-bit divisions, searches: much code, kept in one place)
// and describes them in a ring in shared memory.
struct Part {
  int b, head, pass0, first, count;  // first: among the row's tiles
  int len, nq, lo, hi, tile0, ahead; // as in Span
  int flags;
  int inner_lo, inner_hi;            // every row sees these positions
  static constexpr int kLater = 1, kWhole = 2, kBad = 4, kEnd = 8, kActive = 16;
  __device__ __forceinline__ bool active() const { return kMore ? (flags & kActive) != 0 : hi > lo; }
  __device__ __forceinline__ int pos0(int k) const {
    return (!kMore || first + k < ahead ? tile0 + first + k : first + k - ahead) * kTile;
  }
  __device__ __forceinline__ bool edge(int pos0, int sinks) const {
    return (pos0 < inner_lo && (!kMore || pos0 + kTile > sinks)) || pos0 + kTile > inner_hi;
  }
};
template <int N>
struct Ring {
  const uint32_t base;
  Waiter& w;
  int n = 0;
  __device__ __forceinline__ Ring(uint32_t base_, Waiter& w_) : base(base_), w(w_) {}
  __device__ __forceinline__ Part read(int k) const {
    const uint32_t from = base + Smem<N>::parts + k % kRing * 64;
    const uint4 x = lds128(from), y = lds128(from + 16), z = lds128(from + 32);
    Part p;
    p.b = x.x, p.head = x.y, p.pass0 = x.z, p.first = x.w;
    p.count = __shfl_sync(~0u, y.x, 0), p.len = y.y, p.nq = y.z, p.lo = y.w;
    p.hi = z.x, p.tile0 = z.y, p.flags = z.z, p.inner_lo = z.w;
    p.inner_hi = static_cast<int>(lds32(from + 48));
    p.ahead = kMore ? static_cast<int>(lds32(from + 52)) : 0;
    return p;
  }
  __device__ __forceinline__ void release(int k, int lane) {
    __syncwarp();
    if (lane == 0) w.arrive(kPartEmpty + k % kRing);
  }
  // The next part; false when there is none.
  __device__ __forceinline__ bool next(Part& p, int lane, bool keep = false) {
    w.wait(kPartFull + n % kRing, n / kRing);
    p = read(n);
    if (!keep) release(n, lane);
    ++n;
    return __any_sync(~0u, !w.dead() && !(p.flags & Part::kEnd));
  }
};

// Which rows of a pass see the token at `pos`: [x, y).
template <int N>
__device__ __forceinline__ int2 rows_seeing(const AttnLaunch& L, const Part& p, int pos) {
  const KvAttnArgs& a = L.a;
  if (!in_span(a, p.lo, p.hi, pos)) return make_int2(0, 0);
  // query i sees it if i >= pos - len (its own key included) and i < pos - len + window,
  // or if it is a sink
  const int i = pos - p.len;
  const int lo = a.past_only || i <= 0 ? 0 : i * L.per - p.pass0;
  const long long hi = a.window && !(kMore && pos < a.sinks) ? (static_cast<long long>(i) + a.window) * L.per - p.pass0 : N;
  return make_int2(max(lo, 0), static_cast<int>(max(0ll, min(hi, static_cast<long long>(N)))));
}

// ---- parts and bulk copies (warp 16): eight lanes, a block each ----

template <int N>
__device__ __forceinline__ void copy_role(const AttnLaunch& L, const List<kTile>& list, uint32_t base, Waiter w, int lane) {
  constexpr int S = Smem<N>::kStages;
  const KvAttnArgs& a = L.a;
  const int bpp = a.c.page_size / kKvBlock;
  const long long head_bytes = static_cast<long long>(bpp) * kv_block_bytes(kD), page_bytes = head_bytes * a.c.kv_heads;
  const List<kTile>::Share share = list.share(a, blockIdx.x);
  int left = share.count;
  Place<kTile> place = share.at;
  long long seg = kMore ? blockIdx.x * list.quota - share.row_unit : 0;  // unit of the row's first tile
  if (lane == 0) L.desc[blockIdx.x] = list.parts(share, blockIdx.x);
  int st = 0;
  uint32_t phase = 1;
#pragma unroll 1
  for (int n = 0;; ++n) {
    // the next part (the last says that there are no more)
    Part p;
    p.b = place.b, p.head = place.hr / L.p.rt, p.pass0 = place.hr % L.p.rt * N, p.first = place.tile;
    p.count = min(left, place.s.tiles - place.tile), p.lo = place.s.lo, p.hi = place.s.hi, p.tile0 = place.s.tile0;
    p.ahead = place.s.ahead;
    w.nap(kPartEmpty + n % kRing, (n / kRing) ^ 1);
    if (lane == 0) {
      const uint32_t to = base + Smem<N>::parts + n % kRing * 64;
      const int flags = (n ? Part::kLater : 0) | (p.first == 0 && p.count == place.s.tiles ? Part::kWhole : 0) |
                        (place.s.bad ? Part::kBad : 0) | (left ? 0 : Part::kEnd) | (place.s.any() ? Part::kActive : 0);
      sts128(to, make_uint4(p.b, p.head, p.pass0, p.first));
      sts128(to + 16, make_uint4(p.count, place.s.len, place.s.nq, p.lo));
      sts128(to + 32, make_uint4(p.hi, p.tile0, flags, row_lo(a, place.s, place.s.nq - 1)));
      sts32(to + 48, row_hi(a, place.s.len, 0));
      if (kMore) sts32(to + 52, p.ahead);
      w.arrive(kPartFull + n % kRing);
    }
    if (!left || w.dead()) break;
    const bool any = place.s.any();
    if (own_sums(a) && p.first == 0 && lane == 0)
      a.own_parts[static_cast<long long>(p.b) * list.per_request + place.hr] = list.row_parts(seg, place.s.tiles, blockIdx.x);
    if (kMore) seg += place.s.tiles + list.extra;
    left -= p.count;
    place.tile += p.count - 1;
    if (left) place.next(a, list.per_request);
    if (!any) continue;
    const int32_t* table = a.c.page_table + static_cast<long long>(p.b) * a.c.max_pages;
    const long long head = p.head * head_bytes;
    const auto seen = [&](int k) {
      const int pos = p.pos0(k) + (lane & 7) * kKvBlock;
      return k < p.count && pos < p.hi && (pos + kKvBlock > p.lo || (kMore && pos < a.sinks));
    };
    // the lane's block: its page's column of the table, and its place in the page;
    // page numbers are read a tile ahead
    int col = (p.pos0(0) / kKvBlock + (lane & 7)) / bpp;
    int sub = (p.pos0(0) / kKvBlock + (lane & 7)) - col * bpp;
    bool want = seen(0);
    int page = want ? table[col] : 0;
#pragma unroll 1
    for (int k = 0; k < p.count; ++k) {
      const bool ok = want && page >= 0 && page < a.c.n_pages;
      const int got = __popc(__ballot_sync(~0u, ok) & 0xFFu);
      const bool lacks = (__ballot_sync(~0u, want && !ok) & 0xFFu) != 0;
      const long long at = page * page_bytes + head + static_cast<long long>(sub) * kv_block_bytes(kD);
      sub += kBlocks;
      if (kMore && p.first + k + 1 == p.ahead) {  // on to the sinks
        col = (lane & 7) / bpp;
        sub = (lane & 7) - col * bpp;
      } else if (sub >= bpp) {
        const int q = bpp >= kBlocks ? 1 : sub / bpp;
        col += q;
        sub -= q * bpp;
      }
      const bool want_next = seen(k + 1);
      const int page_next = want_next ? table[col] : 0;
      w.nap(kEmpty + st, phase);
      const uint32_t bar = w.bars + (kFull + st) * 8;
      if (lane == 0) {
        sts32(base + Smem<N>::words + 16 + st * 4, lacks);
        if (lacks) atomicOr(a.status, 1 << SSD_ERR_PAGE);
        bar_expect(bar, got * kv_block_bytes(kD));
      }
      __syncwarp();
      if (lane < 8 && ok && !w.dead())
        bulk_copy(base + Smem<N>::stages + st * kStage + lane * kBlockStride, a.c.pages + at, kv_block_bytes(kD), bar);
      if (++st == S) st = 0, phase ^= 1;
      want = want_next, page = page_next;
    }
  }
  if (w.dead()) {
    // copies still in flight get the same time again before the shared memory goes
    if (lane == 0) atomicOr(a.status, 1 << SSD_ERR_CUDA);
    long long since = 0;
    while (!late(since)) {
    }
  }
}

// ---- queries (warp 19) ----

template <int N>
__device__ __forceinline__ void query_role(const AttnLaunch& L, uint32_t base, Waiter w, int lane) {
  const KvAttnArgs& a = L.a;
  // (strides in elements)
  const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && ((a.qs[0] | a.qs[1] | a.qs[2]) & 7) == 0;
  Ring<N> parts(base, w);
  Part p;
  int n_parts = 0;
  while (parts.next(p, lane)) {
    if (!p.active()) continue;
    const int qb = n_parts & 1, nrows = p.nq * L.per;
    w.nap(kQueryEmpty + qb, (n_parts >> 1) ^ 1);
    // Eight rows at a time, the next eight on their way: a lane has eight elements
    // of every other row.
    const __nv_bfloat16* from =
        static_cast<const __nv_bfloat16*>(a.q) + p.b * a.qs[0] + p.head * L.per * a.qs[2] + (lane & 15) * 8;
    int row = lane >> 4, i = (p.pass0 + row) / L.per, g = (p.pass0 + row) - i * L.per;  // query token and head
    uint4 next[4];
#pragma unroll 1
    for (int k0 = (lane >> 4) - 8; k0 < N; k0 += 8) {
      const uint4 x[4] = {next[0], next[1], next[2], next[3]};
      if (row < N) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          next[k] = make_uint4(0, 0, 0, 0);
          if (p.pass0 + row < nrows) {
            const __nv_bfloat16* q = from + i * a.qs[1] + g * a.qs[2];
            if (vec) {
              next[k] = __ldg(reinterpret_cast<const uint4*>(q));
            } else {
              uint4& v = next[k];
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                const uint32_t h = reinterpret_cast<const unsigned short*>(q)[c];
                v.x = __funnelshift_r(v.x, v.y, 16), v.y = __funnelshift_r(v.y, v.z, 16);
                v.z = __funnelshift_r(v.z, v.w, 16), v.w = __funnelshift_r(v.w, h, 16);
              }
            }
          }
          row += 2;
#pragma unroll 1
          for (g += 2; g >= L.per; g -= L.per) ++i;
        }
      }
      if (k0 < 0) continue;
      // the rows' largest magnitudes: bits of bf16, two of the lane's rows to a word
      uint32_t top[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t m[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint4& v = x[2 * k + y];
          m[y] = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
        }
        top[k] = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
      }
#pragma unroll
      for (int bit = 8; bit; bit >>= 1) {
        top[0] = __vmaxu2(top[0], __shfl_xor_sync(~0u, top[0], bit));
        top[1] = __vmaxu2(top[1], __shfl_xor_sync(~0u, top[1], bit));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // as in ssdv_attn.cu: the row's largest element to [2^12, 2^13), the
        // scale's sign to the query
        int ex = static_cast<int>((k & 1 ? top[k >> 1] >> 16 : top[k >> 1] & 0xFFFFu) >> 7) - 127;
        ex = max(-100, min(ex, 127));
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(12 - ex + 127) << 23), a.scale_log2);
        const int n = k0 + 2 * k;
        const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        uint32_t y[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          y[c] = half2_bits(__floats2half2_rn(__uint_as_float(v[c] << 16) * up, __uint_as_float(v[c] & 0xFFFF0000u) * up));
        sts128(base + Smem<N>::query + qb * Smem<N>::kQueries + operand_byte<N>(n, (lane & 15) * 8),
               make_uint4(y[0], y[1], y[2], y[3]));
        if ((lane & 15) == 0)
          sts_f(base + Smem<N>::factors + (qb * N + n) * 4,
                fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(ex - 12 + 127) << 23));
      }
    }
    async_fence();
    __syncwarp();
    if (lane == 0) w.arrive(kQueryFull + qb);
    ++n_parts;
  }
  if (w.dead() && lane == 0) atomicOr(a.status, 1 << SSD_ERR_CUDA);
}

// ---- matrix instructions (warps 17 and 18; one lane issues them, the warp stays
// together).  An instruction of M = 128 takes 64 cycles or more however few the
// rows, and issuing one waits for those before. ----

// D (+)= A B over 128 of the contraction: A 8 columns a step, B 32 bytes (queries)
// or 16 rows (weights).
template <int N, bool kRowMajor>
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b, bool add, bool leader) {
  // (a broadcast is what tells the compiler that the warp agrees on a number)
  d = __shfl_sync(~0u, d, 0), a = __shfl_sync(~0u, a, 0), b = __shfl_sync(~0u, b, 0);
  const uint64_t operand = tc_operand(b);
#pragma unroll 1
  for (int s = 0; s < 8; ++s)
    tc_mma(d, a + s * 8, operand + (kRowMajor ? s * 128 : (s >> 2) * (N * 8) + (s & 3) * 2), tc_idesc(N, kRowMajor),
           s > 0 || add, leader);
}
// The warp's instructions are done before the tensor memory goes.
__device__ __forceinline__ void drain(const AttnLaunch& L, Waiter& w, bool leader) {
  if (w.dead() && leader) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
  tc_commit(w.bars + kDone * 8, leader);
  bar_wait(w.bars + kDone * 8, 0);
}

template <int N>
__device__ __forceinline__ void score_role(const AttnLaunch& L, uint32_t base, uint32_t tmem, Waiter w, int lane) {
  const bool leader = lane == 0;
  Ring<N> parts(base, w);
  Part p;
  int n_parts = 0, tile = 0;
  while (parts.next(p, lane)) {
    if (!p.active()) continue;
    const int qb = n_parts & 1;
    w.wait(kQueryFull + qb, n_parts >> 1);
#pragma unroll 1
    for (int k = 0; k < p.count; ++k, ++tile) {
      const int sb = tile & 1;
      w.wait(kKeysFull + sb, tile >> 1);
      w.wait(kScoresEmpty + sb, (tile >> 1) ^ 1);
      if (w.dead()) continue;
      tc_fence_after();
      product<N, false>(tmem + Tmem<N>::scores + sb * N, tmem + Tmem<N>::keys + sb * 64,
                        base + Smem<N>::query + qb * Smem<N>::kQueries, false, leader);
      tc_commit(w.bars + (kScoresFull + sb) * 8, leader);
      tc_commit(w.bars + (kKeysEmpty + sb) * 8, leader);
    }
    if (!w.dead()) tc_commit(w.bars + (kQueryEmpty + qb) * 8, leader);
    ++n_parts;
  }
  drain(L, w, leader);
}

template <int N>
__device__ __forceinline__ void sum_role(const AttnLaunch& L, uint32_t base, uint32_t tmem, Waiter w, int lane) {
  const bool leader = lane == 0;
  Ring<N> parts(base, w);
  Part p;
  int n_parts = 0, tile = 0, it = 0, fixes = 0;
  while (parts.next(p, lane)) {
    if (!p.active()) continue;
    const int ob = n_parts % Tmem<N>::kOuts;
    const uint32_t out = tmem + Tmem<N>::outs + ob * N;
    w.wait(kOutEmpty + ob, n_parts / Tmem<N>::kOuts + 1);
#pragma unroll 1
    for (int k = 0; k < p.count; ++k, ++tile) {
      const int vb = tile & 1;
      w.wait(kValuesFull + vb, tile >> 1);
#pragma unroll 1
      for (bool last = false; !last; ++it) {
        const int pb = it & 1;
        w.wait(kWeightsFull + pb, it >> 1);
        const uint32_t info = __shfl_sync(~0u, lds32(base + Smem<N>::words + pb * 4), 0), band = info >> 8;
        last = w.dead() || (info & kInfoLast);
        if (w.dead()) continue;
        if (info & kInfoRescale) {
          // the sums so far are rescaled first
          tc_commit(w.bars + kFixFull * 8, leader);
          w.wait(kFixDone, fixes++);
        }
        tc_fence_after();
        product<N, true>(band ? tmem + Tmem<N>::band : out, tmem + Tmem<N>::values + vb * 64,
                         base + Smem<N>::weight + pb * Smem<N>::kWeights, band == 0 && k > 0, leader);
        tc_commit(w.bars + (kWeightsEmpty + pb) * 8, leader);
        if (band) {
          tc_commit(w.bars + kFixFull * 8, leader);
          w.wait(kFixDone, fixes++);
          tc_fence_after();
        }
        if (last) tc_commit(w.bars + (kValuesEmpty + vb) * 8, leader);
      }
    }
    if (!w.dead()) tc_commit(w.bars + (kOutFull + ob) * 8, leader);
    ++n_parts;
  }
  drain(L, w, leader);
}

// ---- keys (warps 8-11): lane l of warp u has token (l / 4 % 2) + 2 (l / 8) + 8 (u % 2)
// of block l % 4 + 4 (u / 2) ----

template <int N>
__device__ __forceinline__ void key_role(const AttnLaunch& L, uint32_t base, uint32_t tmem, Waiter w, int warp, int lane) {
  constexpr int S = Smem<N>::kStages;
  const Bases bases = make_bases();
  const int blk = (lane & 3) + 4 * (warp >> 1), t = ((lane >> 2) & 1) | ((lane >> 3) << 1) | ((warp & 1) << 3);
  const uint32_t codes = base + Smem<N>::stages + blk * kBlockStride + t * (kD / 2);
  const uint32_t scales = base + Smem<N>::stages + blk * kBlockStride + kv_k_scales(kD) + (t & 1) * 16 + (t >> 1) * 2;
  Ring<N> parts(base, w);
  Part p;
  int st = 0, tile = 0;
  uint32_t phase = 0;
  while (parts.next(p, lane)) {
    if (!p.active()) continue;
#pragma unroll 1
    for (int k = 0; k < p.count; ++k, ++tile) {
      const int kb = tile & 1;
      w.wait(kFull + st, phase);
      const uint32_t from = codes + st * kStage, sfrom = scales + st * kStage;
      w.wait(kKeysEmpty + kb, (tile >> 1) ^ 1);
      tc_fence_after();
      const uint32_t into = tmem + (static_cast<uint32_t>(warp * 32) << 16) + Tmem<N>::keys + kb * 64;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {  // 32 elements, two groups, at a time
        const uint4 c = lds128(from + q * 16);
        const uint32_t word[4] = {c.x, c.y, c.z, c.w}, b = lds16(sfrom + q * 32);
        uint32_t v[16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t s = __byte_perm(b, 0, 0x4040 + 0x0101 * g) << 7;
          const uint32_t s24 = mul2(s, kMinus24), s264 = mul2(s, kMinus264);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int i = g * 2 + x;
            const uint32_t u = __funnelshift_r(word[i], word[i], 8);
            v[4 * i] = fma2(pair_hi(word[i], bases), s, s24);
            v[4 * i + 1] = fma2(pair_lo(word[i], bases), s, s264);
            v[4 * i + 2] = fma2(pair_hi(u, bases), s, s24);
            v[4 * i + 3] = fma2(pair_lo(u, bases), s, s264);
          }
        }
        tc_st16(into + q * 16, v);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        w.arrive(kEmpty + st);
        w.arrive(kKeysFull + kb);
      }
      if (++st == S) st = 0, phase ^= 1;
    }
  }
  if (w.dead() && lane == 0) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
}

// ---- weights (warps 0-7): a thread has one token of the tile, in the keys' order,
// and half of the rows ----

template <int N>
__device__ __forceinline__ void weight_role(const AttnLaunch& L, uint32_t base, uint32_t tmem, Waiter w, int warp, int lane) {
  using M = Smem<N>;
  constexpr int kSync = 1, kThreads = 256, H = N / 2;
  const int tid = warp * 32 + lane, r0 = warp >> 2 ? H : 0;  // its rows begin there
  warp &= 3;
  const int blk = (lane & 3) + 4 * (warp >> 1), t = ((lane >> 2) & 1) | ((lane >> 3) << 1) | ((warp & 1) << 3);
  const int token = blk * kKvBlock + t;
  // In the products' contraction pair p of block b comes at 16 p + 2 b: eight
  // neighbouring lanes then write to different banks.
  const int place = (t >> 1) * 16 + blk * 2 + (t & 1);
  const auto fr_at = [&](int n) { return base + M::fr + (n >> 1) * 16 + (n & 1) * 4; };
  const uint32_t to = base + M::weight + place * 128, turn = (place & 7) << 4;
  Ring<N> parts(base, w);
  Part p;
  int n_parts = 0, tile = 0, it = 0;
  while (parts.next(p, lane)) {
    if (!p.active()) continue;
    const int qb = n_parts & 1;
    w.wait(kQueryFull + qb, n_parts >> 1);
    if (tid < N) {
      sts32(fr_at(tid), lds32(base + M::factors + (qb * N + tid) * 4));
      sts_f(base + M::maxima + tid * 4, -INFINITY);
    }
    group_sync<kThreads>(kSync);
    float l[H];
#pragma unroll
    for (int n = 0; n < H; ++n) l[n] = 0.f;
#pragma unroll 1
    for (int k = 0; k < p.count; ++k, ++tile) {
      const int sb = tile & 1;
      const int pos0 = p.pos0(k);
      const bool edge = p.edge(pos0, L.a.sinks);
      int2 seen = make_int2(0, H);  // which of its rows see the token
      if (edge) {
        seen = rows_seeing<N>(L, p, pos0 + token);
        seen.x -= r0, seen.y -= r0;
      }
      const uint32_t scores = tmem + (static_cast<uint32_t>(warp * 32) << 16) + Tmem<N>::scores + sb * N + r0;
      const auto put = [&](int n, const float* x) {  // its rows n .. n + 7
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = half2_bits(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
        sts128(to + (it & 1) * M::kWeights + (((r0 + n) << 1) ^ turn), make_uint4(v[0], v[1], v[2], v[3]));
      };
      w.wait(kScoresFull + sb, tile >> 1);
      tc_fence_after();
      w.wait(kWeightsEmpty + (it & 1), (it >> 1) ^ 1);
      w.wait(kInfoEmpty + (it & 1), (it >> 1) ^ 1);
      bool rescaled = false;
      int bands = 0;  // passes to come
      float u[H];
#pragma unroll 1
      for (;;) {
        float least = 0.f, most = 0.f;
#pragma unroll
        for (int n = 0; n + 16 <= H; n += 16) tc_ld16(scores + n, u + n);
        if constexpr (H % 16 != 0) tc_ld8(scores + H / 16 * 16, u + H / 16 * 16);
        tc_wait_ld<H>(u);
        const bool first = k == 0 && !rescaled;  // there are no references yet
        if (!first) {
#pragma unroll
          for (int n = 0; n < H; n += 2) {
            const uint4 fr = lds128(base + M::fr + (r0 + n) * 8);  // factors, then references of two rows
            fma_pair(u[n], u[n + 1], fr);
          }
        }
        if (edge) {
#pragma unroll
          for (int n = 0; n < H; ++n) {
            const bool in = n >= seen.x && n < seen.y;
            least = fminf(least, in ? u[n] : 0.f);
            u[n] = in ? u[n] : -INFINITY;
            most = fmaxf(most, u[n]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < H; n += 2) {
            least = fminf(least, fminf(u[n], u[n + 1]));
            most = fmaxf(most, fmaxf(u[n], u[n + 1]));
          }
        }
        const bool high = most > kTop, low = least < kTop - kBand;
        if (!first && !group_any<kThreads>(kSync, high || low)) break;
        if (!first && (rescaled || !group_any<kThreads>(kSync, high))) {
          // below 2^-14 fp16 keeps fewer bits: what it loses goes to later passes
          bands = 1;
          if (!group_any<kThreads>(kSync, least < kTop - 2 * kBand)) break;
          const int need = low ? static_cast<int>(fminf((kTop - least) * (1.f / kBand), kBands - 1.f)) : 0;
          const int most_needed = __reduce_max_sync(~0u, need);
          if (lane == 0 && most_needed)
            atomicMax(reinterpret_cast<int*>(__cvta_shared_to_generic(base + M::words + 8)), most_needed);
          group_sync<kThreads>(kSync);
          bands = lds32(base + M::words + 8);
          group_sync<kThreads>(kSync);
          if (tid == 0) sts32(base + M::words + 8, 0);
          break;
        }
        // the rows' maxima follow the tile's
#pragma unroll 1
        for (int n0 = 0; n0 < H; n0 += 8) {
          float s[8];
          tc_ld8(scores + n0, s);
          tc_wait_ld<8>(s);
          if (edge) {
#pragma unroll
            for (int n = 0; n < 8; ++n) s[n] = n0 + n >= seen.x && n0 + n < seen.y ? s[n] : -INFINITY;
          }
          // rows are exchanged, so that each step halves what a lane holds
#pragma unroll
          for (int half = 4, bit = 16; half; half >>= 1, bit >>= 1) {
            const bool upper = lane & bit;
#pragma unroll
            for (int n = 0; n < half; ++n) {
              const float mine = upper ? s[n + half] : s[n], other = upper ? s[n] : s[n + half];
              s[n] = fmaxf(mine, __shfl_xor_sync(~0u, other, bit));
            }
          }
          s[0] = fmaxf(s[0], __shfl_xor_sync(~0u, s[0], 2));
          s[0] = fmaxf(s[0], __shfl_xor_sync(~0u, s[0], 1));
          if ((lane & 3) == 0) sts_f(base + M::tops + (warp * N + r0 + n0 + (lane >> 2)) * 4, s[0]);
        }
        group_sync<kThreads>(kSync);
        if (tid < N) {
          float top = -INFINITY;
#pragma unroll
          for (int x = 0; x < 4; ++x) top = fmaxf(top, lds_f(base + M::tops + (x * N + tid) * 4));
          const float f = lds_f(fr_at(tid)), old = lds_f(base + M::maxima + tid * 4);
          if (top != -INFINITY) top *= f;
          const float m = fmaxf(old, top);
          sts_f(base + M::maxima + tid * 4, m);
          sts_f(fr_at(tid) + 8, m == -INFINITY ? INFINITY : kFast - m);
          sts_f(base + M::fall + ((it & 1) * N + tid) * 4, old == -INFINITY ? 0.f : ex2(old - m));
        }
        group_sync<kThreads>(kSync);
        if (k > 0) {
#pragma unroll
          for (int n = 0; n < H; ++n) l[n] *= lds_f(base + M::fall + ((it & 1) * N + r0 + n) * 4);
        }
        rescaled = true;
      }
#pragma unroll
      for (int n = 0; n < H; n += 2) {
        u[n] = ex2(u[n]), u[n + 1] = ex2(u[n + 1]);
        add_pair(l[n], l[n + 1], u[n], u[n + 1]);
        if (n % 8 == 6) put(n - 6, u + n - 6);
      }
#pragma unroll 1
      for (int band = 0;; ++band) {
        if (tid == 0)
          sts32(base + M::words + (it & 1) * 4,
                (rescaled && band == 0 && k > 0 ? kInfoRescale : 0) | (band == bands ? kInfoLast : 0) | (band << 8));
        async_fence();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (band == bands) w.arrive(kScoresEmpty + sb);
          w.arrive(kWeightsFull + (it & 1));
        }
        ++it;
        if (band == bands) break;
        w.wait(kWeightsEmpty + (it & 1), (it >> 1) ^ 1);
        w.wait(kInfoEmpty + (it & 1), (it >> 1) ^ 1);
        // what the passes before lost of weights below 2^-14, kBand octaves up each time
        if (band == 0) {
#pragma unroll
          for (int n = 0; n < H; n += 8) {
            float s[8];
#pragma unroll
            for (int y = 0; y < 8; ++y)
              s[y] = u[n + y] < kSmallest ? (u[n + y] - __half2float(__float2half_rn(u[n + y]))) * kBandUp : 0.f;
            put(n, s);
          }
        } else
#pragma unroll 1
        for (int n0 = 0; n0 < H; n0 += 8) {
          float s[8];
          tc_ld8(scores + n0, s);
          tc_wait_ld<8>(s);
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const uint32_t fr = fr_at(r0 + n0 + n);
            s[n] = !edge || (n0 + n >= seen.x && n0 + n < seen.y) ? ex2(fmaf(s[n], lds_f(fr), lds_f(fr + 8))) : 0.f;
          }
#pragma unroll 1
          for (int x = 0; x <= band; ++x)
#pragma unroll
            for (int n = 0; n < 8; ++n)
              s[n] = fabsf(s[n]) < kSmallest ? (s[n] - __half2float(__float2half_rn(s[n]))) * kBandUp : 0.f;
          put(n0, s);
        }
      }
    }
    // the part's sums over the warp's tokens
    const int row = r0 + lane_sums<H, 16>(l, lane);
    constexpr int kLeft = H / ((H & -H) < 32 ? (H & -H) : 32);
    w.wait(kEndEmpty, n_parts ^ 1);
#pragma unroll
    for (int n = 0; n < kLeft; ++n) sts_f(base + M::ends + (warp * N + row + n) * 4, l[n]);
    if (tid < N) sts_f(base + M::ends + (4 * N + tid) * 4, lds_f(base + M::maxima + tid * 4));
    __syncwarp();
    if (lane == 0) {
      w.arrive(kEndFull);
      w.arrive(kQueryEmpty + qb);
    }
    ++n_parts;
    group_sync<kThreads>(kSync);  // the maxima are read before the next part clears them
  }
  if (w.dead() && lane == 0) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
}

// ---- values (warps 12-15): a thread has one element of a head ----

template <int N>
struct Values {
  using M = Smem<N>;
  static constexpr int kSync = 2;
  const AttnLaunch& L;
  const KvAttnArgs& a;
  const uint32_t base, tmem;
  Waiter w;
  const int tid, lane, group, element;
  const Bases bases;
  int it = 0, n_parts = 0, fixes = 0;

  __device__ __forceinline__ Values(const AttnLaunch& L_, uint32_t base_, uint32_t tmem_, Waiter w_, int warp, int lane_)
      : L(L_), a(L_.a), base(base_), tmem(tmem_ + (static_cast<uint32_t>(warp * 32) << 16)), w(w_), tid(warp * 32 + lane_),
        lane(lane_), group((tid >> 1) & 7), element(((tid >> 1) & 7) * 16 + (tid >> 4) * 2 + (tid & 1)), bases(make_bases()) {}

  // A tile's codes to tensor memory.  Returns the rows (bits) that see a NaN among
  // the values of this group in an edge tile, whose other rows must not see it;
  // elsewhere a NaN is every row's.
  __device__ __forceinline__ unsigned long long unpack(int stage, int vb, int tile, int pos0, bool edge, const Part& q) {
    const uint32_t data = base + M::stages + stage * kStage, table = base + M::table + vb * 4096;
    const int blk = tid >> 4, half = tid & 1;  // whose scales this thread expands, for its own group
    uint2 sv = lds64(data + blk * kBlockStride + kv_v_scales(kD) + group * 16 + half * 8);
    if (edge) {
      uint32_t mask = 0;
      const int first = pos0 + blk * kKvBlock + half * 8;
      unsigned long long bytes = sv.x | static_cast<unsigned long long>(sv.y) << 32;
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        const uint32_t byte = static_cast<uint32_t>(bytes >> (k * 8)) & 0xFFu;
        const bool seen = in_span(a, q.lo, q.hi, first + k);
        if (seen && byte == kKvNanByte) mask |= 1u << k;
        if (!seen || byte == kKvNanByte) bytes &= ~(0xFFull << (k * 8));
      }
      sv = make_uint2(static_cast<uint32_t>(bytes), static_cast<uint32_t>(bytes >> 32));
      asm volatile("st.shared.u8 [%0], %1;" ::"r"(base + M::nans + vb * 128 + blk * 16 + group * 2 + half), "r"(mask) : "memory");
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // pairs 4 half + k
      const uint32_t scale = __byte_perm(k < 2 ? sv.x : sv.y, 0, k & 1 ? 0x4342 : 0x4140) << 7;
      sts64(table + (half * 4 + k) * 512 + (blk >> 1) * 128 + group * 16 + (blk & 1) * 8,
            make_uint2(scale, mul2(scale, k & 1 ? kMinus264 : kMinus24)));
    }
    group_sync(kSync);
    w.wait(kValuesEmpty + vb, (tile >> 1) ^ 1);
    tc_fence_after();
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {  // a word of every block, two pairs of it
      uint32_t word[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        word[b] = lds32(data + b * kBlockStride + kv_v_codes(kD) + tid * 8 + (x >> 1) * 4);
        word[b] = __funnelshift_r(word[b], word[b], (x & 1) * 8);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t v[kBlocks];
#pragma unroll
        for (int q = 0; q < kBlocks / 2; ++q) {
          const uint4 e = lds128(table + (x * 2 + k) * 512 + q * 128 + group * 16);
          v[2 * q] = fma2(k ? pair_lo(word[2 * q], bases) : pair_hi(word[2 * q], bases), e.x, e.y);
          v[2 * q + 1] = fma2(k ? pair_lo(word[2 * q + 1], bases) : pair_hi(word[2 * q + 1], bases), e.z, e.w);
        }
        tc_st8(tmem + Tmem<N>::values + vb * 64 + (x * 2 + k) * 8, v);
      }
    }
    unsigned long long rows = 0;
    if (edge) {
#pragma unroll 1
      for (int b = 0; b < kBlocks; ++b) {
        uint32_t nans = lds16(base + M::nans + vb * 128 + b * 16 + group * 2);
#pragma unroll 1
        for (; nans; nans &= nans - 1) {
          const int2 seen = rows_seeing<N>(L, q, pos0 + b * kKvBlock + __ffs(nans) - 1);
          if (seen.x < seen.y) rows |= (~0ull >> (64 - seen.y)) & (~0ull << seen.x);
        }
      }
    }
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      w.arrive(kEmpty + stage);
      w.arrive(kValuesFull + vb);
    }
    return rows;
  }

  // Follows a tile's weights: corrects the sums where the tile asks for it.
  __device__ __forceinline__ void follow() {
#pragma unroll 1
    for (bool last = false; !last; ++it) {
      const int ib = it & 1;
      w.wait(kWeightsFull + ib, it >> 1);
      const uint32_t info = lds32(base + M::words + ib * 4);
      last = w.dead() || (info & kInfoLast);
      const int band = info >> 8;
      if (band || (info & kInfoRescale)) {
        w.wait(kFixFull, fixes++);
        tc_fence_after();
        const uint32_t out = tmem + Tmem<N>::outs + n_parts % Tmem<N>::kOuts * N;
        const float up = band ? ex2(static_cast<float>(-kBand * band)) : 0.f;
#pragma unroll 1
        for (int n = 0; n < N; n += 4) {
          float x[4], t[4];
          tc_ld4(out + n, x);
          tc_ld4(tmem + (band ? Tmem<N>::band + n : Tmem<N>::outs), t);
          tc_wait_ld4(x);
          tc_wait_ld4(t);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            x[y] = band ? fmaf(t[y], up, x[y]) : x[y] * lds_f(base + M::fall + (ib * N + n + y) * 4);
          tc_st4(out + n, x);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) w.arrive(kFixDone);
      }
      __syncwarp();
      if (lane == 0) w.arrive(kInfoEmpty + ib);
    }
  }

  // Writes a part's results; `nans`: rows whose sums a NaN belongs to.
  __device__ __forceinline__ void finish(const Part& q, bool lost, unsigned long long nans) {
    const int nrows = q.flags & Part::kBad ? 0 : q.nq * L.per, ob = n_parts % Tmem<N>::kOuts;
    const bool whole = q.flags & Part::kWhole, active = q.active(), direct = whole && !own_sums(a);
    if ((q.flags & Part::kBad) && q.head == 0 && q.pass0 == 0 && tid == 0) atomicOr(a.status, 1 << SSD_ERR_LENGTH);
    if (active) {
      w.wait(kEndFull, n_parts);
      w.wait(kOutFull + ob, n_parts / Tmem<N>::kOuts);
      tc_fence_after();
    }
    // a thread per row: its factor, and where a whole row goes
    const uint32_t factors = base + M::rows, staged = base + M::results;
    const int live = min(nrows - q.pass0, N);  // rows that are real
    const long long own = (static_cast<long long>(q.b) * a.c.kv_heads + q.head) * L.rows + q.pass0;
    const long long slot = (2ll * blockIdx.x + (q.first == 0 && (q.flags & Part::kLater) ? 1 : 0)) * N;
    __nv_bfloat16* to = nullptr;
    if (tid < N) {
      const int row = q.pass0 + tid;
      float f = 0.f;
      if (row < L.rows && (tid < live || q.first == 0)) {
        const int i = row / L.per;
        const long long orow = (static_cast<long long>(q.b) * a.nq + i) * a.heads + q.head * L.per + row - i * L.per;
        float l = 0.f, m = 0.f;
        if (active && tid < live) {
#pragma unroll
          for (int u = 0; u < 4; ++u) l += lds_f(base + M::ends + (u * N + tid) * 4);
          m = lds_f(base + M::ends + (4 * N + tid) * 4);
        }
        // (a bad page is the queries' own rows' loss, bad lengths are every row's)
        if ((q.flags & Part::kBad) || (tid < live && (lost || w.dead()))) l = __int_as_float(0x7FC00000);
        if (own_sums(a) && (whole || tid >= live)) {
          f = 1 << (kTop - kFast);
          if (tid < live) a.own_ml[own + tid] = make_float2(m, l * f);
        } else if (whole || tid >= live) {
          to = static_cast<__nv_bfloat16*>(a.out) + orow * kD;
          f = l == 0.f ? 0.f : 1.f / l;
          if (a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (m + (log2f(l) - kFast)) * 0.69314718055994531f;
        } else {
          f = 1 << (kTop - kFast);  // (parts are kept 2^kTop up)
          L.ml[slot + tid] = make_float2(m, l * f);
        }
      }
      sts_f(factors + tid * 4, f);
      const uint32_t none = __ballot_sync((tid | 31) < N ? ~0u : 0xFFFFu, f == 0.f);
      if (lane == 0) sts32(factors + (N + warp_of(tid)) * 4, none);
      // the copies of the part before have read what was staged
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    group_sync(kSync);
    unsigned long long none = lds32(factors + N * 4);  // rows whose weights are all zero
    if constexpr (N > 32) none |= static_cast<unsigned long long>(lds32(factors + N * 4 + 4)) << 32;
#pragma unroll 1
    for (int n0 = 0; n0 < N; n0 += 8) {
      float o[8] = {};
      if (active) {
        tc_ld8(tmem + Tmem<N>::outs + ob * N + n0, o);
        tc_wait_ld<8>(o);
      }
      if (none | nans) {
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          if (nans >> (n0 + y) & 1) o[y] = __int_as_float(0x7FC00000);
          if (none >> (n0 + y) & 1) o[y] = 0.f;
        }
      }
      const uint4 fa = lds128(factors + n0 * 4), fb = lds128(factors + n0 * 4 + 16);
      const uint32_t f[8] = {fa.x, fa.y, fa.z, fa.w, fb.x, fb.y, fb.z, fb.w};
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] *= __uint_as_float(f[y]);
      if (direct) {
#pragma unroll
        for (int y = 0; y < 8; y += 2) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(o[y], o[y + 1]);
          const uint32_t x = *reinterpret_cast<const uint32_t*>(&h);
          sts16(staged + (n0 + y) * (kD * 2) + element * 2, x);
          sts16(staged + (n0 + y + 1) * (kD * 2) + element * 2, x >> 16);
        }
      } else {
        float* part = (kMore && whole ? a.own_o + (own + n0) * kD : L.o + (slot + n0) * kD) + element;
#pragma unroll
        for (int y = 0; y < 8; ++y)
          if (n0 + y < live) part[y * kD] = o[y];
      }
    }
    if (direct) {
      async_fence();
      group_sync(kSync);
      if (to)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(staged + tid * (kD * 2)),
                     "n"(kD * 2)
                     : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    } else if (to) {
      // rows past the request's own
      const uint32_t x = q.flags & Part::kBad ? 0x7FC07FC0u : 0u;
      for (int d = 0; d < kD / 8; ++d) reinterpret_cast<uint4*>(to)[d] = make_uint4(x, x, x, x);
    }
    tc_fence_before();
    group_sync(kSync);  // the rows' table is read before the next part's is written
    if (active) {
      if (lane == 0) {
        w.arrive(kEndEmpty);
        w.arrive(kOutEmpty + ob);
      }
      ++n_parts;
    }
  }
};

template <int N>
__device__ __forceinline__ void value_role(const AttnLaunch& L, uint32_t base, uint32_t tmem, Waiter w, int warp, int lane) {
  constexpr int S = Smem<N>::kStages;
  Values<N> v(L, base, tmem, w, warp, lane);
  Ring<N> parts(base, v.w);
  Part p;
  p.count = 0;
  int st = 0, tile = 0, k = 0;
  uint32_t phase = 0;
  // values go one tile ahead of the weights: `pending` of the tile before, whether
  // it was its part's last, and what to know of that part
  bool more = true, pending = false, ends = false, active = false, lost = false, prev_lost = false;
  int prev = 0;
  unsigned long long nans = 0, prev_nans = 0;
#pragma unroll 1
  while (more || pending) {
    if (more && k == p.count) {
      more = parts.next(p, lane, true);  // (kept until its results are written)
      k = 0;
      lost = false;
      nans = 0;
    }
    const bool have = more && p.active();
    if (have) {
      const int pos0 = p.pos0(k);
      v.w.wait(kFull + st, phase);
      lost |= lds32(base + Smem<N>::words + 16 + st * 4) != 0;
      nans |= v.unpack(st, tile & 1, tile, pos0, p.edge(pos0, L.a.sinks), p);
      if (++st == S) st = 0, phase ^= 1;
      ++tile;
    }
    if (pending) {
      // (a part without tiles, whose count is one, has only its results: zeros, or
      // NaN for bad lengths)
      if (active) v.follow();
      if (ends) {
        v.finish(parts.read(prev), prev_lost, prev_nans);
        parts.release(prev, lane);
      }
    }
    pending = more;
    if (more) {
      ++k;
      ends = k == p.count;
      active = have;
      prev = parts.n - 1;
      prev_lost = lost;
      prev_nans = nans;
    }
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  if (v.w.dead() && lane == 0) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tc_kernel(const __grid_constant__ AttnLaunch L) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long scan[kThreads], sums[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem) + 1023) & ~1023u, words = base + Smem<N>::words;
  if (tid < kBars) {
    // how many warps (or commits) arrive
    int count = 1;
    if (tid >= kEmpty && tid < kKeysFull) count = 8;
    if ((tid >= kKeysFull && tid < kKeysEmpty) || (tid >= kValuesFull && tid < kValuesEmpty) ||
        (tid >= kOutEmpty && tid < kQueryFull) || tid == kEndEmpty || tid == kFixDone)
      count = 4;
    if ((tid >= kScoresEmpty && tid < kWeightsEmpty) || tid == kEndFull) count = 8;
    if (tid >= kQueryEmpty && tid < kEndFull) count = 9;
    if (tid == kDone) count = 2;
    if (tid >= kPartEmpty) count = 19;
    bar_init(base + tid * 8, count);
  }
  if (tid < kMaxStages) sts32(words + 16 + tid * 4, 0);
  if (tid == 0) sts32(words + 8, 0);
  if (warp == 17) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(words + 12) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  tc_fence_before();
  if constexpr (kMore) asm volatile("griddepcontrol.wait;" ::: "memory");
  List<kTile> list;
  list.build(L.a, L.a.c.kv_heads * L.p.rt, gridDim.x, kPartTiles, scan, sums);
  tc_fence_after();
  const uint32_t tmem = lds32(words + 12);
  Waiter w;
  w.bars = base;
  // 128 x (112 + 112 + 72 + 96 + 88) registers: the 640 x 96 of the launch
  if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
  else if (warp < 12) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  else if (warp >= 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  // Their code lies in this order: the three that work all the time share the
  // instruction cache best side by side (64 requests of 201 to 8003 tokens, 20
  // rows: 102 us; with the values' code before the keys' 118).
  if (warp < 8) weight_role<N>(L, base, tmem, w, warp, lane);
  else if (warp >= 8 && warp < 12) key_role<N>(L, base, tmem, w, warp - 8, lane);
  else if (warp >= 12 && warp < 16) value_role<N>(L, base, tmem, w, warp - 12, lane);
  else if (warp == 18) sum_role<N>(L, base, tmem, w, lane);
  else if (warp == 17) score_role<N>(L, base, tmem, w, lane);
  else if (warp == 16) copy_role<N>(L, list, base, w, lane);
  else if (warp == 19) query_role<N>(L, base, w, lane);
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int N>
cudaError_t launch_n(const AttnLaunch& L, int sms, cudaStream_t stream) {
  const cudaError_t e = allow_shared<kv_attention_tc_kernel<N>>(Smem<N>::total);
  if (e != cudaSuccess) return e;
  if constexpr (kMore) return launch_after(kv_attention_tc_kernel<N>, dim3(sms), kThreads, Smem<N>::total, stream, L);
  kv_attention_tc_kernel<N><<<sms, kThreads, Smem<N>::total, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace

#if SSDV_ATTN_MORE
cudaError_t launch_attention_tc_more(const AttnLaunch& L, int sms, cudaStream_t stream) {
#else
cudaError_t launch_attention_tc(const AttnLaunch& L, int sms, cudaStream_t stream) {
#endif
  switch (L.rows_pass) {
    case 32: return launch_n<32>(L, sms, stream);
    case 48: return launch_n<48>(L, sms, stream);
    case 64: return launch_n<64>(L, sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ssdv
