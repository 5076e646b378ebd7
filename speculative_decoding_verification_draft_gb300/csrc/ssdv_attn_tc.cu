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
// Sixteen warps with one job each, joined by mbarriers:
//   0-3   weights: scores from tensor memory, softmax, weights to shared memory
//   4-7   keys: codes to tensor memory
//   8-11  values: codes to tensor memory; then each tile's product is added to
//         the fp32 sums in registers with its rows' factors
//   12    bulk copies of the tiles' blocks   13  issues the matrix instructions
//   14-15 queries
// Every buffer is double, so that a tile's scores, the tile before's weights and
// the values of both overlap.
//
// Weights are fp16, 2^(x - m + kFast) with m the row's maximum so far, while all
// of a tile's lie in [2^-14, 2^15], where fp16 keeps 11 bits; then the tile's
// product is simply added.  Otherwise the tile takes its own maximum (at 2^15)
// and a factor, and the weights below 2^-14 are passed over again, kBand octaves
// a pass, as in ssdv_attn.cu.
#include "ssdv_attn.cuh"

#include <algorithm>

namespace ssdv {

namespace {

constexpr int kTile = 128;
constexpr int kBlocks = kTile / kKvBlock;
constexpr int kD = 128;
constexpr int kThreads = 512;
constexpr int kFast = 9, kTop = 15;
constexpr int kMaxStages = 8;
// Blocks lie 16 bytes past a multiple of 128 apart: the eight lanes of a phase,
// four blocks' two tokens, then read different banks.
constexpr int kBlockStride = kv_block_bytes(kD) + 16;
constexpr int kStage = kBlocks * kBlockStride;
constexpr int kHead = 1024;
constexpr int kSmem = 227000;

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
  kSumFull = 32,        // [2] product computed         -> values
  kSumEmpty = 34,       // [2] product read             -> matrix
  kInfoEmpty = 36,      // [2] factors read             -> weights
  kQueryFull = 38,      // [2] queries written          -> matrix, weights
  kQueryEmpty = 40,     // [2] queries done with        -> queries
  kEndFull = 42,        // a part's sums of weights     -> values
  kEndEmpty = 43,       // read                         -> weights
  kDone = 44,           // all matrix instructions are done
  kBars = 45
};

// Shared memory after the head, for N rows.
template <int N>
struct Smem {
  static constexpr int kOperand = N * 256;  // N rows x 128 fp16, 128-byte swizzled halves
  static constexpr int query = kHead;
  static constexpr int weight = query + 2 * kOperand;
  static constexpr int table = weight + 2 * kOperand;   // [2] scales of the values: 8 blocks x 4 x 8 groups x 16 bytes
  static constexpr int nans = table + 2 * 4096;         // [2][8 blocks][8 groups][2] bytes
  static constexpr int fr = nans + 2 * 128;             // [N] factor and reference of the fast weights
  static constexpr int maxima = fr + 8 * N;             // [N]
  static constexpr int tops = maxima + 4 * N;           // [4][N]
  static constexpr int refs = tops + 16 * N;            // [N] references of a tile's own weights
  static constexpr int gaps = refs + 4 * N;             // [N] tile's maximum below the row's
  static constexpr int grow = gaps + 4 * N;             // [2][N]
  static constexpr int fall = grow + 8 * N;             // [2][N]
  static constexpr int factors = fall + 8 * N;          // [2][N]
  static constexpr int spans = factors + 8 * N;         // [2][N] int2
  static constexpr int ends = spans + 16 * N;           // [4][N] sums, [N] maxima
  static constexpr int words = ends + 20 * N;           // info [2], bands, tensor memory address, flags [8]
  static constexpr int stages = (words + 64 + 127) / 128 * 128;
  static constexpr int kStages = (kSmem - stages) / kStage < kMaxStages ? (kSmem - stages) / kStage : kMaxStages;
  static constexpr int total = stages + kStages * kStage + 1024;  // the operands begin at a multiple of 1024
};
constexpr int kInfoSlow = 1, kInfoLast = 2;

// Tensor memory columns: keys and values twice 64 (128 fp16 a lane), scores twice
// N, products once or twice N.
template <int N>
struct Tmem {
  static constexpr int keys = 0, values = 128, scores = 256, sums = 256 + 2 * N;
  static constexpr int kSums = N <= 64 ? 2 : 1;
  static_assert(sums + kSums * N <= 512, "tensor memory");
};

// ---- tcgen05 ----

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 16 columns of the warp's 32 lanes; not to be used before tc_wait_ld.
__device__ __forceinline__ void tc_ld16(uint32_t at, float* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]),
        "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
      : "r"(at));
}
// Waits for the loads; the registers pass through, so that no use moves ahead.
template <int N>
__device__ __forceinline__ void tc_wait_ld(float* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i += 16)
    asm volatile(""
                 : "+f"(x[i]), "+f"(x[i + 1]), "+f"(x[i + 2]), "+f"(x[i + 3]), "+f"(x[i + 4]), "+f"(x[i + 5]),
                   "+f"(x[i + 6]), "+f"(x[i + 7]), "+f"(x[i + 8]), "+f"(x[i + 9]), "+f"(x[i + 10]), "+f"(x[i + 11]),
                   "+f"(x[i + 12]), "+f"(x[i + 13]), "+f"(x[i + 14]), "+f"(x[i + 15]));
}
__device__ __forceinline__ void tc_st32(uint32_t at, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// D [128 x N] in tensor memory (+)= A [128 x 16] in tensor memory, B [N x 16] in shared memory.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// fp16 x fp16 -> fp32, both operands contraction-major, M = 128.
__device__ __forceinline__ constexpr uint32_t tc_idesc(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n / 8) << 17) | ((128u / 16) << 24);
}
// An operand of 128-byte rows, 128-byte swizzle: 8-row groups lie 1024 bytes apart.
__device__ __forceinline__ uint64_t tc_operand(uint32_t at) {
  return (static_cast<uint64_t>(at >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Byte of element (row, column) of such an operand of N x 128 fp16 in two halves.
template <int N>
__device__ __forceinline__ uint32_t operand_byte(int row, int column) {
  return static_cast<uint32_t>((column >> 6) * (N * 128) + row * 128 + ((((column >> 3) & 7) ^ (row & 7)) << 4) +
                               (column & 7) * 2);
}

__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "bar.red.or.pred p, %1, 128, q;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float lds_f(uint32_t p) { return __uint_as_float(lds32(p)); }
__device__ __forceinline__ void sts_f(uint32_t p, float x) { sts32(p, __float_as_uint(x)); }
__device__ __forceinline__ void sts16(uint32_t p, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(p), "h"(static_cast<unsigned short>(v)) : "memory");
}
__device__ __forceinline__ uint32_t lds16(uint32_t p) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p));
  return v;
}
// The larger of all lanes' numbers (NaN aside).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(y) : "f"(x));
  return y;
}

// Waits that end: once one has run out, the warp goes through the motions
// without waiting, so that every barrier of the CTA is still met.
struct Waiter {
  uint32_t bars;
  bool dead = false;
  __device__ __forceinline__ void wait(int bar, uint32_t phase) {
    if (!dead && !bar_wait(bars + bar * 8, phase & 1)) dead = true;
  }
  __device__ __forceinline__ void arrive(int bar) { bar_arrive(bars + bar * 8); }
};

// A CTA's share of the list, part by part: tiles of one (request, head, pass).
struct Part {
  int b, hr, first, count;
  bool later;  // not the first of the CTA's
  Span s;
  __device__ __forceinline__ bool active() const { return s.hi > s.lo; }
};
struct Parts {
  const KvAttnArgs& a;
  const List<kTile>& list;
  Place<kTile> at;
  int left;
  bool begun = false;
  __device__ __forceinline__ Parts(const KvAttnArgs& a_, const List<kTile>& l) : a(a_), list(l) {
    const long long u = blockIdx.x * l.quota;
    left = u < l.units ? static_cast<int>(min(l.units - u, l.quota)) : 0;
    if (left) at = l.find(a, u);
  }
  __device__ __forceinline__ bool next(Part& p) {
    if (!left) return false;
    p.b = at.b, p.hr = at.hr, p.first = at.tile, p.s = at.s;
    p.count = min(left, at.s.tiles - at.tile);
    p.later = begun;
    begun = true;
    left -= p.count;
    at.tile += p.count - 1;
    if (left) at.next(a, list.per_request);
    return true;
  }
};

// ---- bulk copies (warp 12): eight lanes, a block each ----

template <int N>
__device__ __forceinline__ void copy_role(const AttnLaunch& L, const List<kTile>& list, uint32_t base, Waiter w, int lane) {
  constexpr int S = Smem<N>::kStages;
  const KvAttnArgs& a = L.a;
  const int bpp = a.c.page_size / kKvBlock;
  const long long head_bytes = static_cast<long long>(bpp) * kv_block_bytes(kD), page_bytes = head_bytes * a.c.kv_heads;
  Parts parts(a, list);
  Part p;
  int st = 0;
  uint32_t phase = 1;
  while (parts.next(p)) {
    if (!p.active()) continue;
    const int32_t* table = a.c.page_table + static_cast<long long>(p.b) * a.c.max_pages;
    const long long head = p.hr / L.p.rt * head_bytes;
    const auto column = [&](int k) { return ((p.s.tile0 + p.first + k) * kBlocks + (lane & 7)) / bpp; };
    const auto seen = [&](int k) {
      const int pos = (p.s.tile0 + p.first + k) * kTile + (lane & 7) * kKvBlock;
      return k < p.count && pos < p.s.hi && pos + kKvBlock > p.s.lo;
    };
    // page numbers are read a tile ahead
    bool want = seen(0);
    int col = column(0), page = want ? table[col] : 0;
    for (int k = 0; k < p.count; ++k) {
      const int sub = (p.s.tile0 + p.first + k) * kBlocks + (lane & 7) - col * bpp;
      const bool ok = want && page >= 0 && page < a.c.n_pages;
      const int got = __popc(__ballot_sync(~0u, ok) & 0xFFu);
      const bool lacks = (__ballot_sync(~0u, want && !ok) & 0xFFu) != 0;
      const long long at = page * page_bytes + head + static_cast<long long>(sub) * kv_block_bytes(kD);
      const bool want_next = seen(k + 1);
      const int col_next = column(k + 1), page_next = want_next ? table[col_next] : 0;
      w.wait(kEmpty + st, phase);
      const uint32_t bar = w.bars + (kFull + st) * 8;
      if (lane == 0) {
        sts32(base + Smem<N>::words + 16 + st * 4, lacks);
        if (lacks) atomicOr(a.status, 1 << SSD_ERR_PAGE);
        bar_expect(bar, got * kv_block_bytes(kD));
      }
      __syncwarp();
      if (lane < 8 && ok && !w.dead)
        bulk_copy(base + Smem<N>::stages + st * kStage + lane * kBlockStride, a.c.pages + at, kv_block_bytes(kD), bar);
      if (++st == S) st = 0, phase ^= 1;
      want = want_next, col = col_next, page = page_next;
    }
  }
  if (w.dead) {
    // copies still in flight get the same time again before the shared memory goes
    if (lane == 0) atomicOr(a.status, 1 << SSD_ERR_CUDA);
    unsigned long long since = 0;
    while (!late(since)) {
    }
  }
}

// ---- queries (warps 14, 15): every other row each ----

template <int N>
__device__ __forceinline__ void query_role(const AttnLaunch& L, const List<kTile>& list, uint32_t base, Waiter w, int warp,
                                           int lane) {
  const KvAttnArgs& a = L.a;
  Parts parts(a, list);
  Part p;
  int n = 0;
  while (parts.next(p)) {
    if (!p.active()) continue;
    const int qb = n & 1;
    w.wait(kQueryEmpty + qb, (n >> 1) ^ 1);
    const int h = p.hr / L.p.rt, pass0 = p.hr % L.p.rt * N, nrows = p.s.nq * L.per;
#pragma unroll 4
    for (int k = warp; k < N; k += 2) {
      const int row = pass0 + k;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (row < nrows) {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + p.b * a.qs[0] + row / L.per * a.qs[1] +
                                 (h * L.per + row % L.per) * a.qs[2] + lane * 4;
        if ((reinterpret_cast<uintptr_t>(q) & 7) == 0) {
          const uint2 v = *reinterpret_cast<const uint2*>(q);
          x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
          x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = static_cast<float>(q[e]);
        }
      }
      float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
      top = warp_max(top);
      // as in ssdv_attn.cu: the row's largest element to [2^12, 2^13), the
      // scale's sign to the query
      int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      ex = max(-100, min(ex, 127));
      const float up = copysignf(__uint_as_float(static_cast<uint32_t>(12 - ex + 127) << 23), a.scale_log2);
      const uint32_t at = base + Smem<N>::query + qb * Smem<N>::kOperand + operand_byte<N>(k, lane * 4);
      sts64(at, make_uint2(half2_bits(__floats2half2_rn(x[0] * up, x[1] * up)),
                           half2_bits(__floats2half2_rn(x[2] * up, x[3] * up))));
      if (lane == 0) {
        sts_f(base + Smem<N>::factors + (qb * N + k) * 4,
              fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(ex - 12 + 127) << 23));
        const int i = row / L.per;
        sts64(base + Smem<N>::spans + (qb * N + k) * 8,
              make_uint2(row_lo(a, p.s.len, i), min(row_hi(a, p.s.len, i), p.s.hi)));
      }
    }
    async_fence();
    __syncwarp();
    if (lane == 0) w.arrive(kQueryFull + qb);
    ++n;
  }
  if (w.dead && lane == 0) atomicOr(a.status, 1 << SSD_ERR_CUDA);
}

// ---- matrix instructions (one thread) ----

template <int N>
__device__ __forceinline__ void matrix_role(const AttnLaunch& L, const List<kTile>& list, uint32_t base, uint32_t tmem,
                                            Waiter w) {
  constexpr uint32_t idesc = tc_idesc(N);
  Parts parts(L.a, list);
  Part p;
  p.count = 0;
  int in_part = 0, n_parts = 0, scored = 0;
  // scores of the next tile, if there is one
  const auto scores = [&]() -> bool {
    while (in_part == p.count) {
      if (!parts.next(p)) return false;
      in_part = p.active() ? 0 : p.count;
    }
    const int sb = scored & 1, qb = n_parts & 1;
    if (in_part == 0) w.wait(kQueryFull + qb, n_parts >> 1);
    w.wait(kKeysFull + sb, scored >> 1);
    w.wait(kScoresEmpty + sb, (scored >> 1) ^ 1);
    tc_fence_after();
    if (!w.dead) {
#pragma unroll
      for (int s = 0; s < 8; ++s)
        tc_mma(tmem + Tmem<N>::scores + sb * N, tmem + Tmem<N>::keys + sb * 64 + s * 8,
               tc_operand(base + Smem<N>::query + qb * Smem<N>::kOperand + (s >> 2) * (N * 128) + (s & 3) * 32), idesc,
               s > 0);
      tc_commit(w.bars + (kScoresFull + sb) * 8);
      tc_commit(w.bars + (kKeysEmpty + sb) * 8);
    }
    ++scored;
    if (++in_part == p.count) {
      if (!w.dead) tc_commit(w.bars + (kQueryEmpty + qb) * 8);
      ++n_parts;
    }
    return true;
  };
  int tile = 0, it = 0;
  bool more = scores();
  while (more) {
    more = scores();
    const int vb = tile & 1;
    for (bool first = true, last = false; !last; first = false) {
      const int pb = it & 1, tb = it % Tmem<N>::kSums;
      if (first) w.wait(kValuesFull + vb, tile >> 1);
      w.wait(kWeightsFull + pb, it >> 1);
      w.wait(kSumEmpty + tb, it / Tmem<N>::kSums + 1);
      last = w.dead || (lds32(base + Smem<N>::words + pb * 4) & kInfoLast);
      tc_fence_after();
      if (!w.dead) {
#pragma unroll
        for (int s = 0; s < 8; ++s)
          tc_mma(tmem + Tmem<N>::sums + tb * N, tmem + Tmem<N>::values + vb * 64 + s * 8,
                 tc_operand(base + Smem<N>::weight + pb * Smem<N>::kOperand + (s >> 2) * (N * 128) + (s & 3) * 32), idesc,
                 s > 0);
        tc_commit(w.bars + (kSumFull + tb) * 8);
        tc_commit(w.bars + (kWeightsEmpty + pb) * 8);
        if (last) tc_commit(w.bars + (kValuesEmpty + vb) * 8);
      }
      ++it;
    }
    ++tile;
  }
  if (w.dead) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
  tc_commit(w.bars + kDone * 8);
  bar_wait(w.bars + kDone * 8, 0);
}

// ---- keys (warps 4-7): lane l of warp u has token (l / 4 % 2) + 2 (l / 8) + 8 (u % 2)
// of block l % 4 + 4 (u / 2) ----

template <int N>
__device__ __forceinline__ void key_role(const AttnLaunch& L, const List<kTile>& list, uint32_t base, uint32_t tmem, Waiter w,
                                         int warp, int lane) {
  constexpr int S = Smem<N>::kStages;
  const Bases bases = make_bases();
  const int blk = (lane & 3) + 4 * (warp >> 1), t = ((lane >> 2) & 1) | ((lane >> 3) << 1) | ((warp & 1) << 3);
  const uint32_t codes = base + Smem<N>::stages + blk * kBlockStride + t * (kD / 2);
  const uint32_t scales = base + Smem<N>::stages + blk * kBlockStride + kv_k_scales(kD) + (t & 1) * 16 + (t >> 1) * 2;
  Parts parts(L.a, list);
  Part p;
  int st = 0, tile = 0;
  uint32_t phase = 0;
  while (parts.next(p)) {
    if (!p.active()) continue;
    for (int k = 0; k < p.count; ++k, ++tile) {
      const int kb = tile & 1;
      w.wait(kFull + st, phase);
      const uint32_t from = codes + st * kStage, sfrom = scales + st * kStage;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 c0 = lds128(from + half * 32), c1 = lds128(from + half * 32 + 16);
        const uint32_t word[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        uint32_t v[32];
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          const uint32_t b = lds16(sfrom + (half * 2 + g2) * 32);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint32_t s = __byte_perm(b, 0, 0x4040 + 0x0101 * g) << 7;
            const uint32_t s24 = mul2(s, kMinus24), s264 = mul2(s, kMinus264);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int i = g2 * 4 + g * 2 + x;
              const uint32_t u = __funnelshift_r(word[i], word[i], 8);
              v[4 * i] = fma2(pair_hi(word[i], bases), s, s24);
              v[4 * i + 1] = fma2(pair_lo(word[i], bases), s, s264);
              v[4 * i + 2] = fma2(pair_hi(u, bases), s, s24);
              v[4 * i + 3] = fma2(pair_lo(u, bases), s, s264);
            }
          }
        }
        if (half == 0) {
          w.wait(kKeysEmpty + kb, (tile >> 1) ^ 1);
          tc_fence_after();
        }
        tc_st32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + Tmem<N>::keys + kb * 64 + half * 32, v);
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
  if (w.dead && lane == 0) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
}

// ---- weights (warps 0-3): a thread has one token of the tile, the keys' order ----

template <int N>
__device__ __forceinline__ void weight_role(const AttnLaunch& L, const List<kTile>& list, uint32_t base, uint32_t tmem,
                                            Waiter w, int warp, int lane) {
  using M = Smem<N>;
  constexpr int kSync = 1;
  const int tid = warp * 32 + lane;
  const int token = ((lane & 3) + 4 * (warp >> 1)) * kKvBlock + (((lane >> 2) & 1) | ((lane >> 3) << 1) | ((warp & 1) << 3));
  const uint32_t scores = tmem + (static_cast<uint32_t>(warp * 32) << 16) + Tmem<N>::scores;
  uint32_t to[8];  // where the thread's column of the weights lies in rows 0..7
#pragma unroll
  for (int r = 0; r < 8; ++r) to[r] = base + M::weight + operand_byte<N>(r, token);
  Parts parts(L.a, list);
  Part p;
  int n_parts = 0, tile = 0, it = 0;
  while (parts.next(p)) {
    if (!p.active()) continue;
    const int qb = n_parts & 1;
    w.wait(kQueryFull + qb, n_parts >> 1);
    if (tid < N) {
      // an infinite reference makes the first tile take its own
      sts64(base + M::fr + tid * 8, make_uint2(lds32(base + M::factors + (qb * N + tid) * 4), 0x7F800000u));
      sts_f(base + M::maxima + tid * 4, -INFINITY);
    }
    group_sync(kSync);
    const int lo_last = row_lo(L.a, p.s.len, p.s.nq - 1), hi_first = row_hi(L.a, p.s.len, 0);
    float l[N];
#pragma unroll
    for (int n = 0; n < N; ++n) l[n] = 0.f;
    for (int k = 0; k < p.count; ++k, ++tile) {
      const int sb = tile & 1;
      const int pos0 = (p.s.tile0 + p.first + k) * kTile, pos = pos0 + token;
      const bool edge = pos0 < lo_last || pos0 + kTile > hi_first;
      float s[N];
      const auto load = [&]() {
#pragma unroll
        for (int n = 0; n < N; n += 16) tc_ld16(scores + sb * N + n, s + n);
        tc_wait_ld<N>(s);
        if (edge) {
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const uint2 seen = lds64(base + M::spans + (qb * N + n) * 8);
            if (pos < static_cast<int>(seen.x) || pos >= static_cast<int>(seen.y)) s[n] = -INFINITY;
          }
        }
      };
      const auto put = [&](int n, uint32_t pair) {
        sts16(to[n & 7] + (it & 1) * M::kOperand + (n >> 3) * 1024, pair);
        sts16(to[(n + 1) & 7] + (it & 1) * M::kOperand + (n >> 3) * 1024, pair >> 16);
      };
      w.wait(kScoresFull + sb, tile >> 1);
      tc_fence_after();
      load();
      w.wait(kWeightsEmpty + (it & 1), (it >> 1) ^ 1);
      bool out = false;
      __half2 least = __float2half2_rn(1.f), most = least;
#pragma unroll
      for (int n = 0; n < N; n += 2) {
        const uint4 fr = lds128(base + M::fr + n * 8);
        const float e0 = ex2(fmaf(s[n], __uint_as_float(fr.x), __uint_as_float(fr.y)));
        const float e1 = ex2(fmaf(s[n + 1], __uint_as_float(fr.z), __uint_as_float(fr.w)));
        if (edge) {
          const bool seen0 = s[n] != -INFINITY, seen1 = s[n + 1] != -INFINITY;
          s[n] = seen0 ? e0 : 0.f, s[n + 1] = seen1 ? e1 : 0.f;
          out |= (seen0 && (e0 < kSmallest || e0 > 32768.f)) || (seen1 && (e1 < kSmallest || e1 > 32768.f));
          put(n, half2_bits(__floats2half2_rn(s[n], s[n + 1])));
        } else {
          s[n] = e0, s[n + 1] = e1;
          const __half2 h = __floats2half2_rn(e0, e1);
          least = __hmin2(least, h);
          most = __hmax2(most, h);
          put(n, half2_bits(h));
        }
      }
      if (!edge)
        out = __low2float(least) < kSmallest || __high2float(least) < kSmallest || __low2float(most) > 32768.f ||
              __high2float(most) > 32768.f;
      if (!group_any(kSync, out)) {
#pragma unroll
        for (int n = 0; n < N; ++n) l[n] += s[n];
        w.wait(kInfoEmpty + (it & 1), (it >> 1) ^ 1);
        if (tid == 0) sts32(base + M::words + (it & 1) * 4, kInfoLast);
        async_fence();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          w.arrive(kScoresEmpty + sb);
          w.arrive(kWeightsFull + (it & 1));
        }
        ++it;
        continue;
      }
      // the tile's own maxima
      load();
      float keep[(N + 31) / 32];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float top = warp_max(s[n]);
        if (lane == (n & 31)) keep[n >> 5] = top;
      }
#pragma unroll
      for (int j = 0; j < (N + 31) / 32; ++j)
        if (j * 32 + lane < N) sts_f(base + M::tops + (warp * N + j * 32 + lane) * 4, keep[j]);
      w.wait(kInfoEmpty + (it & 1), (it >> 1) ^ 1);
      group_sync(kSync);
      if (tid < N) {
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < 4; ++u) top = fmaxf(top, lds_f(base + M::tops + (u * N + tid) * 4));
        const float f = lds_f(base + M::fr + tid * 8), old = lds_f(base + M::maxima + tid * 4);
        if (top != -INFINITY) top *= f;
        const float m = fmaxf(old, top), zero = m == -INFINITY ? 0.f : m;
        if (top == -INFINITY) top = zero;
        sts_f(base + M::maxima + tid * 4, m);
        sts_f(base + M::fr + tid * 8 + 4, m == -INFINITY ? INFINITY : kFast - m);
        sts_f(base + M::refs + tid * 4, kTop - top);
        sts_f(base + M::gaps + tid * 4, top - zero);
        sts_f(base + M::grow + ((it & 1) * N + tid) * 4, ex2(top - zero + (kFast - kTop)));
        sts_f(base + M::fall + ((it & 1) * N + tid) * 4, ex2(old - zero));
      }
      if (tid == 0) sts32(base + M::words + 8, 0);
      group_sync(kSync);
      uint32_t bands = 0;
      for (uint32_t todo = 1; todo;) {
        const int band = __ffs(todo) - 1;
        todo &= todo - 1;
        const int ib = it & 1;
        if (band) {
          w.wait(kWeightsEmpty + ib, (it >> 1) ^ 1);
          w.wait(kInfoEmpty + ib, (it >> 1) ^ 1);
          if (tid < N) {
            sts_f(base + M::grow + (ib * N + tid) * 4,
                  ex2(lds_f(base + M::gaps + tid * 4) + (kFast - kTop - kBand * band)));
            sts_f(base + M::fall + (ib * N + tid) * 4, 1.f);
          }
        }
#pragma unroll
        for (int n = 0; n < N; n += 2) {
          uint32_t pair = 0;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float u = fmaf(s[n + x], lds_f(base + M::fr + (n + x) * 8), lds_f(base + M::refs + (n + x) * 4));
            int at = u >= kTop - kBand ? 0 : min(kBands, static_cast<int>((kTop - u) * (1.f / kBand)));
            const bool seen = !edge || s[n + x] != -INFINITY;
            if (!seen) at = kBands;
            if (band == 0) {
              const float e = seen ? ex2(u) : 0.f;
              l[n + x] = l[n + x] * lds_f(base + M::fall + (ib * N + n + x) * 4) +
                         e * lds_f(base + M::grow + (ib * N + n + x) * 4);
              if (at > 0 && at < kBands) bands |= 1u << at;
            }
            const float e = at == band ? ex2(u + kBand * band) : 0.f;
            pair |= static_cast<uint32_t>(__half_as_ushort(__float2half_rn(e))) << (16 * x);
          }
          put(n, pair);
        }
        if (band == 0) {
          bands = __reduce_or_sync(~0u, bands);
          if (lane == 0 && bands) atomicOr(reinterpret_cast<uint32_t*>(__cvta_shared_to_generic(base + M::words + 8)), bands);
          group_sync(kSync);
          todo = lds32(base + M::words + 8);
        }
        if (tid == 0) sts32(base + M::words + ib * 4, kInfoSlow | (todo ? 0 : kInfoLast));
        async_fence();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!todo) w.arrive(kScoresEmpty + sb);
          w.arrive(kWeightsFull + ib);
        }
        ++it;
      }
    }
    // the part's sums over the warp's tokens: pairs of rows are exchanged, so
    // that each step halves what a lane holds
    int width = N, row = 0;
#pragma unroll
    for (int bit = 16; bit; bit >>= 1) {
      if (width % 2 == 0) {
        const int half = width / 2;
        const bool upper = lane & bit;
#pragma unroll
        for (int n = 0; n < N / 2; ++n)
          if (n < half) {
            const float mine = upper ? l[n + half] : l[n], other = upper ? l[n] : l[n + half];
            l[n] = mine + __shfl_xor_sync(~0u, other, bit);
          }
        row += upper ? half : 0;
        width = half;
      } else {
#pragma unroll
        for (int n = 0; n < N / 2; ++n)
          if (n < width) l[n] += __shfl_xor_sync(~0u, l[n], bit);
      }
    }
    w.wait(kEndEmpty, n_parts ^ 1);
#pragma unroll
    for (int n = 0; n < N / 2; ++n)
      if (n < width) sts_f(base + M::ends + (warp * N + row + n) * 4, l[n]);
    if (tid < N) sts_f(base + M::ends + (4 * N + tid) * 4, lds_f(base + M::maxima + tid * 4));
    __syncwarp();
    if (lane == 0) {
      w.arrive(kEndFull);
      w.arrive(kQueryEmpty + qb);
    }
    ++n_parts;
    group_sync(kSync);  // the maxima are read before the next part clears them
  }
  if (w.dead && lane == 0) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
}

// ---- values (warps 8-11): a thread has one element of a head ----

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
  float o[N];
  int it = 0, n_parts = 0;
  uint32_t nans[4] = {};  // tokens of the pending tile whose values of this group are NaN

  __device__ __forceinline__ Values(const AttnLaunch& L_, uint32_t base_, uint32_t tmem_, Waiter w_, int warp, int lane_)
      : L(L_), a(L_.a), base(base_), tmem(tmem_ + (static_cast<uint32_t>(warp * 32) << 16)), w(w_), tid(warp * 32 + lane_),
        lane(lane_), group((tid >> 1) & 7), element(((tid >> 1) & 7) * 16 + (tid >> 4) * 2 + (tid & 1)), bases(make_bases()) {
#pragma unroll
    for (int n = 0; n < N; ++n) o[n] = 0.f;
  }

  // A tile's codes to tensor memory; `found`: its NaN (edge tiles, whose other
  // rows must not see them; elsewhere a NaN is every row's).
  __device__ __forceinline__ void unpack(int stage, int vb, int tile, int pos0, bool edge, const Span& sp,
                                         uint32_t (&found)[4]) {
    const uint32_t data = base + M::stages + stage * kStage, table = base + M::table + vb * 4096;
    const int blk = tid >> 4, half = tid & 1;  // whose scales this thread expands, for its own group
    uint2 sv = lds64(data + blk * kBlockStride + kv_v_scales(kD) + group * 16 + half * 8);
    if (edge) {
      uint32_t mask = 0;
      uint32_t sc[2] = {sv.x, sv.y};
      const int first = pos0 + blk * kKvBlock + half * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t byte = (sc[k >> 2] >> ((k & 3) * 8)) & 0xFFu;
        const bool seen = first + k >= sp.lo && first + k < sp.hi;
        if (seen && byte == kKvNanByte) mask |= 1u << k;
        if (!seen || byte == kKvNanByte) sc[k >> 2] &= ~(0xFFu << ((k & 3) * 8));
      }
      sv = make_uint2(sc[0], sc[1]);
      asm volatile("st.shared.u8 [%0], %1;" ::"r"(base + M::nans + vb * 128 + blk * 16 + group * 2 + half), "r"(mask) : "memory");
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t word = k ? sv.y : sv.x;
      const uint32_t s0 = __byte_perm(word, 0, 0x4140) << 7, s1 = __byte_perm(word, 0, 0x4342) << 7;
      sts128(table + blk * 512 + half * 256 + k * 128 + group * 16,
             make_uint4(s0, mul2(s0, kMinus24), s1, mul2(s1, kMinus264)));
    }
    group_sync(kSync);
    w.wait(kValuesEmpty + vb, (tile >> 1) ^ 1);
    tc_fence_after();
#pragma unroll
    for (int quad = 0; quad < 2; ++quad) {
      uint32_t v[32];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint2 c = lds64(data + (quad * 4 + b) * kBlockStride + kv_v_codes(kD) + tid * 8);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t word = k ? c.y : c.x, turned = __funnelshift_r(word, word, 8);
          const uint4 e0 = lds128(table + (quad * 4 + b) * 512 + (2 * k) * 128 + group * 16);
          const uint4 e1 = lds128(table + (quad * 4 + b) * 512 + (2 * k + 1) * 128 + group * 16);
          v[b * 8 + k * 4] = fma2(pair_hi(word, bases), e0.x, e0.y);
          v[b * 8 + k * 4 + 1] = fma2(pair_lo(word, bases), e0.z, e0.w);
          v[b * 8 + k * 4 + 2] = fma2(pair_hi(turned, bases), e1.x, e1.y);
          v[b * 8 + k * 4 + 3] = fma2(pair_lo(turned, bases), e1.z, e1.w);
        }
      }
      tc_st32(tmem + Tmem<N>::values + vb * 64 + quad * 32, v);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) found[x] = 0;
    if (edge)
#pragma unroll
      for (int b = 0; b < 8; ++b) found[b >> 1] |= lds16(base + M::nans + vb * 128 + b * 16 + group * 2) << (16 * (b & 1));
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      w.arrive(kEmpty + stage);
      w.arrive(kValuesFull + vb);
    }
  }

  // Adds the products of a tile that began at pos0.
  __device__ __forceinline__ void gather(const Part& q, int pos0) {
    if (nans[0] | nans[1] | nans[2] | nans[3]) {
      const int pass0 = q.hr % L.p.rt * N;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int i = (pass0 + n) / L.per;
        const int lo = max(0, min(row_lo(a, q.s.len, i) - pos0, kTile));
        const int hi = max(0, min(min(row_hi(a, q.s.len, i), q.s.hi) - pos0, kTile));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int from = max(0, min(lo - 32 * x, 32)), to = max(0, min(hi - 32 * x, 32));
          const uint32_t below = to == 32 ? ~0u : (1u << to) - 1u, skip = from == 32 ? ~0u : (1u << from) - 1u;
          if (nans[x] & below & ~skip) o[n] = __int_as_float(0x7FC00000);
        }
      }
    }
    __syncwarp();
    for (bool last = false; !last;) {
      const int tb = it % Tmem<N>::kSums, ib = it & 1;
      w.wait(kSumFull + tb, it / Tmem<N>::kSums);
      tc_fence_after();
      const uint32_t info = lds32(base + M::words + ib * 4);
      last = w.dead || (info & kInfoLast);
#pragma unroll
      for (int n = 0; n < N; n += 16) {
        float t[16];
        tc_ld16(tmem + Tmem<N>::sums + tb * N + n, t);
        tc_wait_ld<16>(t);
        if (info & kInfoSlow) {
#pragma unroll
          for (int y = 0; y < 16; ++y)
            o[n + y] = o[n + y] * lds_f(base + M::fall + (ib * N + n + y) * 4) +
                       t[y] * lds_f(base + M::grow + (ib * N + n + y) * 4);
        } else {
#pragma unroll
          for (int y = 0; y < 16; ++y) o[n + y] += t[y];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        w.arrive(kSumEmpty + tb);
        w.arrive(kInfoEmpty + ib);
      }
      ++it;
    }
  }

  // Writes a part's results and clears the sums.
  __device__ __forceinline__ void finish(const Part& q, bool lost) {
    const int h = q.hr / L.p.rt, pass0 = q.hr % L.p.rt * N;
    const int nrows = q.s.bad ? 0 : q.s.nq * L.per;
    const bool whole = q.first == 0 && q.count == q.s.tiles, active = q.active();
    const long long slot = 2ll * blockIdx.x + (q.first == 0 && q.later ? 1 : 0);
    if (q.s.bad && q.hr == 0 && tid == 0) atomicOr(a.status, 1 << SSD_ERR_LENGTH);
    if (active) w.wait(kEndFull, n_parts);
    lost = lost || w.dead || q.s.bad;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int row = pass0 + n;
      if (row < L.rows) {
        const long long orow = (static_cast<long long>(q.b) * a.nq + row / L.per) * a.heads + h * L.per + row % L.per;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + orow * kD + element;
        float l = 0.f, m = 0.f;
        if (active) {
#pragma unroll
          for (int u = 0; u < 4; ++u) l += lds_f(base + M::ends + (u * N + n) * 4);
          m = lds_f(base + M::ends + (4 * N + n) * 4);
        }
        if (row >= nrows) l = 0.f;  // a padded query's row
        if (lost) l = __int_as_float(0x7FC00000);
        if (row >= nrows ? q.first == 0 : whole) {
          *out = static_cast<__nv_bfloat16>(l == 0.f ? 0.f : o[n] / l);
          if (a.lse && tid == 0) a.lse[orow] = l == 0.f ? -INFINITY : (m + (log2f(l) - kFast)) * 0.69314718055994531f;
        } else if (row < nrows) {
          // (parts are kept 2^kTop up)
          const long long at = slot * N + n;
          L.o[at * kD + element] = o[n] * (1 << (kTop - kFast));
          if (tid == 0) L.ml[at] = make_float2(m, l * (1 << (kTop - kFast)));
        }
      }
      o[n] = 0.f;
    }
    if (active) {
      __syncwarp();
      if (lane == 0) w.arrive(kEndEmpty);
      ++n_parts;
    }
  }
};

template <int N>
__device__ __forceinline__ void value_role(const AttnLaunch& L, const List<kTile>& list, uint32_t base, uint32_t tmem,
                                           Waiter w, int warp, int lane) {
  constexpr int S = Smem<N>::kStages;
  Values<N> v(L, base, tmem, w, warp, lane);
  Parts parts(L.a, list);
  Part p, prev = {};
  int st = 0, tile = 0, prev_pos0 = 0;
  uint32_t phase = 0;
  // a tile's products are added while the next one's are computed
  bool pending = false, ends = false, lost = false, prev_lost = false;
  while (parts.next(p)) {
    if (!p.active()) {
      if (pending) {
        v.gather(prev, prev_pos0);
        v.finish(prev, prev_lost);
        pending = false;
      }
      v.finish(p, false);
      continue;
    }
    const int lo_last = row_lo(L.a, p.s.len, p.s.nq - 1), hi_first = row_hi(L.a, p.s.len, 0);
    lost = false;
    for (int k = 0; k < p.count; ++k, ++tile) {
      const int pos0 = (p.s.tile0 + p.first + k) * kTile;
      uint32_t found[4];
      v.w.wait(kFull + st, phase);
      lost |= lds32(base + Smem<N>::words + 16 + st * 4) != 0;
      v.unpack(st, tile & 1, tile, pos0, pos0 < lo_last || pos0 + kTile > hi_first, p.s, found);
      if (++st == S) st = 0, phase ^= 1;
      if (pending) {
        v.gather(prev, prev_pos0);
        if (ends) v.finish(prev, prev_lost);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) v.nans[x] = found[x];
      pending = true;
      ends = k == p.count - 1;
      prev = p;
      prev_pos0 = pos0;
      prev_lost = lost;
    }
  }
  if (pending) {
    v.gather(prev, prev_pos0);
    v.finish(prev, prev_lost);
  }
  if (v.w.dead && lane == 0) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tc_kernel(const __grid_constant__ AttnLaunch L) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long scan[kThreads], sums[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem) + 1023) & ~1023u, words = base + Smem<N>::words;
  if (tid < kBars) {
    int count = 1;
    if (tid >= kEmpty && tid < kKeysFull) count = 8;
    if ((tid >= kKeysFull && tid < kKeysEmpty) || (tid >= kScoresEmpty && tid < kWeightsEmpty) ||
        (tid >= kValuesFull && tid < kValuesEmpty) || (tid >= kSumEmpty && tid < kQueryFull) || tid >= kEndFull)
      count = 4;
    if (tid >= kQueryFull && tid < kQueryEmpty) count = 2;
    if (tid >= kQueryEmpty && tid < kEndFull) count = 5;
    if (tid == kDone) count = 1;
    bar_init(base + tid * 8, count);
  }
  if (tid < kMaxStages) sts32(words + 16 + tid * 4, 0);
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(words + 12) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  tc_fence_before();
  List<kTile> list;
  list.build(L.a, L.a.c.kv_heads * L.p.rt, gridDim.x, scan, sums);
  tc_fence_after();
  const uint32_t tmem = lds32(words + 12);
  Waiter w;
  w.bars = base;
  // 128 x (192 + 96 + 152 + 72) registers: the 512 x 128 of the launch
  if (warp < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    weight_role<N>(L, list, base, tmem, w, warp, lane);
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    key_role<N>(L, list, base, tmem, w, warp - 4, lane);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    value_role<N>(L, list, base, tmem, w, warp - 8, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 12) {
      copy_role<N>(L, list, base, w, lane);
    } else if (warp == 13) {
      if (lane == 0) matrix_role<N>(L, list, base, tmem, w);
      __syncwarp();
    } else {
      if (warp == 14 && lane == 0) {
        const long long me = blockIdx.x;
        L.desc[me] = me * list.quota < list.units ? list.parts(list.find(L.a, me * list.quota), me) : make_int4(0, 0, 0, 0);
      }
      query_role<N>(L, list, base, w, warp - 14, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int N>
cudaError_t launch_n(const AttnLaunch& L, int sms, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(kv_attention_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Smem<N>::total);
  if (e != cudaSuccess) return e;
  kv_attention_tc_kernel<N><<<sms, kThreads, Smem<N>::total, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_tc(const AttnLaunch& L, int sms, cudaStream_t stream) {
  switch (L.rows_pass) {
    case 16: return launch_n<16>(L, sms, stream);
    case 32: return launch_n<32>(L, sms, stream);
    case 48: return launch_n<48>(L, sms, stream);
    case 64: return launch_n<64>(L, sms, stream);
    case 80: return launch_n<80>(L, sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ssdv
