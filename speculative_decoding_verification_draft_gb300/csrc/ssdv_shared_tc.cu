// ssdv_shared_tc.cu -- attention over a shared prefix on the fifth-generation tensor
// cores: bf16 queries, 64 or 128 elements a head.
//
// Rows are the M side here (a group has hundreds of them): 256 rows of a row block,
// two tiles of 128, meet tiles of 128 tokens, scored in halves.
//   S [128 rows x 64 tokens]     = Q K^T     both operands in shared memory
//   O [128 rows x D elements]   += P V       P in tensor memory
// Keys and values are unpacked once for all 256 rows, to fp16, where n s is exact.
//
// Twenty warps:
//   0-3, 4-7   weights of the first and the second 128 rows, a thread a row: maximum,
//              2^x, sum, weights back to tensor memory, corrections, results
//   8-11       keys: a token a thread, from global memory to a shared operand
//   12-15      values: two elements of some blocks a thread, likewise
//   16, 17     issue the matrix instructions of the first and the second 128 rows
//   18         finds the CTA's parts of the list
// Scores go to registers as soon as they are there, so the next half's are computed
// while this half's weights are; weights of two halves are kept, so that no matrix
// instruction waits for another's end.
//
// Weights are fp16, 2^(x - m + 9), with m the row's maximum when it was last moved:
// first taken from a part's first tile, it moves when a tile's weights add up to more
// than fp16 holds, so most tiles are passed over once, without a maximum, and sums are
// corrected a few times a row.  fp16 keeps 11 bits down to 2^-14, 23 octaves below m,
// and multiples of 2^-24 below that; an error of half of one is 2^-34 of the row's
// largest weight at most.  Outputs are bf16.  Maxima, sums of weights and of values are
// fp32.
#include "ssdv_shared.cuh"
#include "ssdv_tc.cuh"

namespace ssdv {

namespace {

constexpr int kTile = 128, kM = 128, kThreads = 640;
constexpr int kHalf = 64;  // tokens that are scored at a time
constexpr int kFast = 9, kTop = 15;

enum : int {
  kKeysFull = 0,      // [2] keys unpacked               -> matrix
  kKeysEmpty = 2,     // [2] both tiles' scores computed -> keys
  kValuesFull = 4,    // [2] values unpacked             -> matrix
  kValuesEmpty = 6,   // [2] both tiles' products        -> values
  kQueryFull = 8,     // [2 tiles of rows] queries written       -> matrix
  kScoresFull = 10,   // [2] half a tile's scores computed       -> weights
  kScoresRead = 12,   // [2] and in registers                    -> matrix
  kWeightsFull = 14,  // [2][2] weights written, sums corrected  -> matrix
  kOutFull = 18,      // [2][2] half a tile's products added     -> weights
  kDone = 22,         // all matrix instructions are done
  kPartFull = 23,     // [kRing] a part is described          -> all
  kPartEmpty = 27,    // [kRing] all have read it             -> plan
  kPlaceFull = 31,    // [kPlaces] a tile's blocks are found  -> keys, values
  kPlaceEmpty = 39,   // [kPlaces] both have read them        -> plan
  kBars = 47
};
constexpr int kRing = 4, kReaders = 18, kPlaces = 8;
constexpr int kTmemAt = 384, kPartsAt = 512, kPlacesAt = 768;  // bytes; a part 64, a tile's eight blocks 64

template <int D>
struct Smem {
  static constexpr int kOperand = kTile * D * 2;  // 128 rows or tokens x D, or D x 128
  static constexpr int query = 2048, keys = query + 2 * kOperand, values = keys + 2 * kOperand;
  static constexpr int total = values + 2 * kOperand + 1024;  // operands begin at a multiple of 1024
};
// Columns of tensor memory: each tile of rows' scores of half a tile, weights of two
// halves (two fp16 a column), sums.
constexpr int kScoresAt = 0, kWeightsAt = 2 * kHalf, kOutAt = 4 * kHalf;

__device__ __forceinline__ void tc_ld32(uint32_t at, float (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
      "%31}, [%32];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]),
        "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(x[16]),
        "=f"(x[17]), "=f"(x[18]), "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]),
        "=f"(x[25]), "=f"(x[26]), "=f"(x[27]), "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31])
      : "r"(at));
}
// D [128 x N] in tensor memory (+)= A [128 x 16] B [N x 16], both in shared memory.
__device__ __forceinline__ void tc_mma_shared(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, bool leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(leader))
      : "memory");
}

// A role's view of the CTA.  Parts are found by one warp (64-bit divisions, searches)
// and described in a ring in shared memory.
struct Roles {
  const SharedLaunch& L;
  uint32_t base, tmem;
  Waiter w;
  int n = 0;
  // The CTA's next part, false when there is none.
  __device__ __forceinline__ bool next(SharedPart& p, int lane) {
    w.wait(kPartFull + n % kRing, n / kRing);
    const uint32_t from = base + kPartsAt + n % kRing * 64;
    const uint4 x = lds128(from), y = lds128(from + 16);
    const uint2 z = lds64(from + 32);
    p.h = x.x, p.block = x.y, p.b0 = x.z, p.n_rows = x.w;
    p.len = y.x, p.t0 = y.y, p.count = __shfl_sync(~0u, y.z, 0);
    p.row0 = z.x | static_cast<long long>(z.y) << 32;
    __syncwarp();
    if (lane == 0) w.arrive(kPartEmpty + n % kRing);
    ++n;
    return __any_sync(~0u, !w.dead() && p.count > 0);
  }
};
__device__ __forceinline__ void part_role(const SharedLaunch& L, const GroupList& list, uint32_t base, Waiter w, int lane,
                                          int block_bytes) {
  const KvCacheArgs& c = L.a.c;
  const int bpp = c.page_size / kKvBlock;
  long long u = blockIdx.x * list.quota;
  const long long end = min(u + list.quota, list.total);
  int it = 0;
  bool bad = false;
#pragma unroll 1
  for (int n = 0; !w.dead(); ++n) {
    SharedPart p = {};
    if (u < end) p = list.part(u, end);
    u += p.count;
    w.nap(kPartEmpty + n % kRing, (n / kRing) ^ 1);
    if (lane == 0) {
      const uint32_t to = base + kPartsAt + n % kRing * 64;
      sts128(to, make_uint4(p.h, p.block, p.b0, p.n_rows));
      sts128(to + 16, make_uint4(p.len, p.t0, p.count, 0));
      sts64(to + 32, make_uint2(static_cast<uint32_t>(p.row0), static_cast<uint32_t>(p.row0 >> 32)));
      w.arrive(kPartFull + n % kRing);
    }
    if (p.count == 0) break;
    // where the tiles' blocks lie (null behind the prefix and on a bad page): eight
    // lanes, a block each, pages a tile ahead
    const int32_t* table = c.page_table + static_cast<long long>(p.b0) * c.max_pages;
    int at = p.t0 * 8 + (lane & 7), col = at / bpp, sub = at - col * bpp;
    const auto page_of = [&]() { return at * kKvBlock < p.len ? table[col] : -1; };
    int page = page_of();
#pragma unroll 1
    for (int k = 0; k < p.count; ++k, ++it) {
      const bool there = at * kKvBlock < p.len, ok = there && page >= 0 && page < c.n_pages;
      bad |= there && !ok;
      const uint8_t* from =
          ok ? c.pages + ((static_cast<long long>(page) * c.kv_heads + p.h) * bpp + sub) * block_bytes : nullptr;
      at += 8, sub += 8;
      if (sub >= bpp) {
        const int q = bpp >= 8 ? 1 : sub / bpp;
        col += q;
        sub -= q * bpp;
      }
      if (k + 1 < p.count) page = page_of();
      const int slot = it % kPlaces;
      w.nap(kPlaceEmpty + slot, (it / kPlaces) ^ 1);
      if (lane < 8) {
        const unsigned long long v = reinterpret_cast<unsigned long long>(from);
        sts64(base + kPlacesAt + slot * 64 + lane * 8, make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32)));
      }
      __syncwarp();
      if (lane == 0) w.arrive(kPlaceFull + slot);
    }
  }
  if (bad) atomicOr(L.a.status, 1 << SSD_ERR_PAGE);
  if (w.dead() && lane == 0) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
}

__device__ __forceinline__ const uint8_t* pointer(uint32_t lo, uint32_t hi) {
  return reinterpret_cast<const uint8_t*>(lo | static_cast<unsigned long long>(hi) << 32);
}

// ---- keys ----

template <int D>
__device__ __forceinline__ void key_role(Roles r, int tid) {
  constexpr int kWords = D / 32;  // 16 bytes of codes
  const int lane = tid & 31, t = tid & 15, blk = tid >> 4;
  const Bases bases = make_bases();
  // chunk c of 8 elements of row `tid` lies at c ^ (tid & 7) of its 128 bytes
  const uint32_t to = r.base + Smem<D>::keys + tid * 128 + ((tid & 7) << 4);
  uint4 c[kWords];
  uint32_t s[kWords];  // two groups' scales each
  const uint8_t* from;
  const auto find = [&](int it) {
    const int slot = it % kPlaces;
    r.w.wait(kPlaceFull + slot, it / kPlaces);
    const uint2 v = lds64(r.base + kPlacesAt + slot * 64 + blk * 8);
    from = pointer(v.x, v.y);
    __syncwarp();
    if (lane == 0) r.w.arrive(kPlaceEmpty + slot);
  };
  const auto load = [&](int i) {  // 32 elements; NaN where there is no block
    c[i] = from ? __ldg(reinterpret_cast<const uint4*>(from + k_word_offset<D>(t, i * 4))) : make_uint4(0, 0, 0, 0);
    if constexpr (D == 64) {
      s[i] = from ? __ldg(from + k_scale_offset<D>(t, 2 * i)) | __ldg(from + k_scale_offset<D>(t, 2 * i + 1)) << 8 : 0xFFFFu;
    } else {
      s[i] = from ? __ldg(reinterpret_cast<const unsigned short*>(from + k_scale_offset<D>(t, 2 * i))) : 0xFFFFu;
    }
  };
  SharedPart p;
  int it = 0;
  while (r.next(p, lane)) {
    find(it);
#pragma unroll
    for (int i = 0; i < kWords; ++i) load(i);
#pragma unroll 1
    for (int k = 0; k < p.count; ++k, ++it) {
      const bool more = k + 1 < p.count;
      if (more) find(it + 1);
      const int st = it & 1;
      r.w.wait(kKeysEmpty + st, (it >> 1) ^ 1);
      const uint32_t row = to + st * Smem<D>::kOperand;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t words[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        // what is behind the prefix may be anything: its scores are not used
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t x = __byte_perm(s[i], 0, g ? 0x4141 : 0x4040) << 7;
          const uint32_t x24 = mul2(x, kMinus24), x264 = mul2(x, kMinus264);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t v = words[g * 2 + y], u = __funnelshift_r(v, v, 8);
            const int chunk = i * 4 + g * 2 + y;  // of 8 elements
            sts128((row ^ ((chunk & 7) << 4)) + (chunk >> 3) * (kTile * 128),
                   make_uint4(fma2(pair_hi(v, bases), x, x24), fma2(pair_lo(v, bases), x, x264),
                              fma2(pair_hi(u, bases), x, x24), fma2(pair_lo(u, bases), x, x264)));
          }
        }
        if (more) load(i);
      }
      async_fence();
      __syncwarp();
      if (lane == 0) r.w.arrive(kKeysFull + st);
    }
  }
  if (r.w.dead() && lane == 0) atomicOr(r.L.a.status, 1 << SSD_ERR_CUDA);
}

// ---- values: lane l has elements (2 i, 2 i + 1) of row g of the codes' order, i = l %
// (D / 16), and half of the lanes take them the other way round, so that eight
// neighbours write to different banks ----

template <int D>
__device__ __forceinline__ void value_role(Roles r, int tid) {
  constexpr int kI = D / 16, kB = D / 32;  // blocks a thread
  const int lane = tid & 31, warp = tid >> 5, i = lane & (kI - 1), swap = (lane >> 2) & 1;
  const int g = lane / kI + (D == 128 ? 4 * (warp & 1) : 0), b0 = (D == 128 ? warp >> 1 : warp) * kB;
  const int d0 = g * (D / 8) + 2 * i;
  const Bases bases = make_bases();
  // chunk c of 8 tokens of row d lies at c ^ (d & 7) of its 128 bytes
  uint32_t to[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int d = d0 + (e ^ swap);
    to[e] = (r.base + Smem<D>::values + d * 128 + ((d & 7) << 4)) ^ ((b0 & 3) << 5);
    if (b0 & 4) to[e] += D * 128;
  }
  uint4 c[kB], s[kB];
  uint32_t at[2 * kB];  // where the next tile's blocks are
  const auto find = [&](int it) {
    const int slot = it % kPlaces;
    r.w.wait(kPlaceFull + slot, it / kPlaces);
#pragma unroll
    for (int b = 0; b < kB; b += 2) {
      const uint4 v = lds128(r.base + kPlacesAt + slot * 64 + (b0 + b) * 8);
      at[2 * b] = v.x, at[2 * b + 1] = v.y, at[2 * b + 2] = v.z, at[2 * b + 3] = v.w;
    }
    __syncwarp();
    if (lane == 0) r.w.arrive(kPlaceEmpty + slot);
  };
  const auto load = [&](int b) {
    const uint8_t* from = pointer(at[2 * b], at[2 * b + 1]);
    c[b] = from ? __ldg(reinterpret_cast<const uint4*>(from + v_word_offset<D>(d0, 0))) : make_uint4(0, 0, 0, 0);
    s[b] = from ? __ldg(reinterpret_cast<const uint4*>(from + kv_v_scales(D) + (d0 >> 4) * 16)) : make_uint4(0, 0, 0, 0);
  };
  SharedPart p;
  int it = 0;
  while (r.next(p, lane)) {
    find(it);
#pragma unroll
    for (int b = 0; b < kB; ++b) load(b);
#pragma unroll 1
    for (int k = 0; k < p.count; ++k, ++it) {
      const int st = it & 1, pos0 = (p.t0 + k) * kTile;
      const bool more = k + 1 < p.count;
      if (more) find(it + 1);
      if (pos0 + kTile > p.len) {
        // tokens behind the prefix: zero
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const int seen = p.len - pos0 - (b0 + b) * 16;
          const auto keep = [&](uint32_t v, int x) {
            return seen >= 4 * x + 4 ? v : seen <= 4 * x ? 0u : v & ((1u << (seen - 4 * x) * 8) - 1u);
          };
          s[b] = make_uint4(keep(s[b].x, 0), keep(s[b].y, 1), keep(s[b].z, 2), keep(s[b].w, 3));
        }
      }
      r.w.wait(kValuesEmpty + st, (it >> 1) ^ 1);
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const uint32_t sb[4] = {s[b].x, s[b].y, s[b].z, s[b].w};
        const uint4 code = c[b];
        if (more) load(b);
        const uint32_t first[2] = {swap ? code.z : code.x, swap ? code.x : code.z};
        const uint32_t second[2] = {swap ? code.w : code.y, swap ? code.y : code.w};
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // 8 tokens
          uint32_t x[4], o[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            x[y] = __byte_perm(sb[half * 2 + (y >> 1)], 0, y & 1 ? 0x4342 : 0x4140) << 7;
            o[y] = mul2(x[y], y & 1 ? kMinus264 : kMinus24);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t v = half ? second[e] : first[e], u = __funnelshift_r(v, v, 8);
            sts128((to[e] ^ ((b * 2 + half) << 4)) + st * Smem<D>::kOperand,
                   make_uint4(fma2(pair_hi(v, bases), x[0], o[0]), fma2(pair_lo(v, bases), x[1], o[1]),
                              fma2(pair_hi(u, bases), x[2], o[2]), fma2(pair_lo(u, bases), x[3], o[3])));
          }
        }
      }
      async_fence();
      __syncwarp();
      if (lane == 0) r.w.arrive(kValuesFull + st);
    }
  }
  if (r.w.dead() && lane == 0) atomicOr(r.L.a.status, 1 << SSD_ERR_CUDA);
}

// ---- matrix instructions of a tile of rows (one lane issues them) ----

template <int D>
__device__ __forceinline__ void matrix_role(Roles r, int tile, int lane) {
  const bool leader = lane == 0;
  const uint32_t scores = r.tmem + kScoresAt + tile * kHalf, weights = r.tmem + kWeightsAt + tile * kHalf;
  const uint32_t out = r.tmem + kOutAt + tile * D;
  const uint64_t query = tc_operand(r.base + Smem<D>::query + tile * Smem<D>::kOperand);
  const uint64_t keys = tc_operand(r.base + Smem<D>::keys), values = tc_operand(r.base + Smem<D>::values);
  Waiter& w = r.w;
  // scores of half h of the tile in stage st
  const auto score = [&](int st, int h) {
    if (w.dead()) return;
    tc_fence_after();
#pragma unroll 1
    for (int s = 0; s < D / 16; ++s) {
      const int at = (s >> 2) * (kTile * 128 / 16) + (s & 3) * 2;
      tc_mma_shared(scores, query + at, keys + st * (Smem<D>::kOperand / 16) + h * (kHalf * 128 / 16) + at,
                    tc_idesc(kHalf, false), s > 0, leader);
    }
    tc_commit(w.bars + (kScoresFull + tile) * 8, leader);
    if (h) tc_commit(w.bars + (kKeysEmpty + st) * 8, leader);
  };
  SharedPart p;
  int it = 0, mine = 0, parts = 0;
  while (r.next(p, lane)) {
    if (tile && p.n_rows <= kM) {
      // nothing to do with this part's tiles but to let them go
#pragma unroll 1
      for (int k = 0; k < p.count; ++k, ++it) {
        w.wait(kKeysFull + (it & 1), it >> 1);
        if (leader) w.arrive(kKeysEmpty + (it & 1));
        w.wait(kValuesFull + (it & 1), it >> 1);
        if (leader) w.arrive(kValuesEmpty + (it & 1));
      }
      continue;
    }
    w.wait(kQueryFull + tile, parts++);
    w.wait(kKeysFull + (it & 1), it >> 1);
    score(it & 1, 0);
#pragma unroll 1
    for (int k = 0; k < 2 * p.count; ++k, ++mine) {
      const int h = k & 1, st = it & 1;
      // the next half's scores, once these have been read
      if (h && k + 1 < 2 * p.count) w.wait(kKeysFull + (st ^ 1), (it + 1) >> 1);
      w.wait(kScoresRead + tile, mine);
      if (k + 1 < 2 * p.count) score(h ? st ^ 1 : st, h ^ 1);
      if (h == 0) w.wait(kValuesFull + st, it >> 1);
      w.wait(kWeightsFull + tile * 2 + h, mine >> 1);
      if (!w.dead()) {
        tc_fence_after();
#pragma unroll 1
        for (int s = 0; s < kHalf / 16; ++s)
          tc_mma(out, weights + h * (kHalf / 2) + s * 8,
                 values + st * (Smem<D>::kOperand / 16) + h * (D * 128 / 16) + s * 2, tc_idesc(D, false), k > 0 || s > 0,
                 leader);
        tc_commit(w.bars + (kOutFull + tile * 2 + h) * 8, leader);
        if (h) tc_commit(w.bars + (kValuesEmpty + st) * 8, leader);
      }
      it += h;
    }
  }
  if (w.dead() && leader) atomicOr(r.L.a.status, 1 << SSD_ERR_CUDA);
  tc_commit(w.bars + kDone * 8, leader);
  bar_wait(w.bars + kDone * 8, 0);
}

// ---- weights: a thread a row ----

template <int D>
__device__ __forceinline__ void weight_role(Roles r, int tile, int tid) {
  const SharedLaunch& L = r.L;
  const int lane = tid & 31;
  const uint32_t lanes = static_cast<uint32_t>(tid & 96) << 16;
  const uint32_t scores = r.tmem + lanes + kScoresAt + tile * kHalf;
  const uint32_t weights = r.tmem + lanes + kWeightsAt + tile * kHalf, out = r.tmem + lanes + kOutAt + tile * D;
  const uint32_t query = r.base + Smem<D>::query + tile * Smem<D>::kOperand + tid * 128;
  const bool vec =
      (reinterpret_cast<uintptr_t>(L.a.q) & 15) == 0 && ((L.a.qs[0] | L.a.qs[1] | L.a.qs[2]) & 7) == 0;  // (in elements)
  Waiter& w = r.w;
  SharedPart p;
  int mine = 0;
  while (r.next(p, lane)) {
    if (tile && p.n_rows <= kM) continue;
    const int row = tile * kM + tid;
    float f;
    {
      // the query as fp16, a power of two up: its largest element to [2^12, 2^13), the
      // scale's sign on it (exact down to 2^-26 of the largest)
      const SharedRow at(L, p, row);
      const unsigned short* q =
          static_cast<const unsigned short*>(L.a.q) + at.b * L.a.qs[0] + at.i * L.a.qs[1] + at.head * L.a.qs[2];
      const auto load = [&](int c) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (at.real) {
          if (vec) {
            v = __ldg(reinterpret_cast<const uint4*>(q) + c);
          } else {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
              const uint32_t h = q[c * 8 + e];
              v.x = __funnelshift_r(v.x, v.y, 16), v.y = __funnelshift_r(v.y, v.z, 16);
              v.z = __funnelshift_r(v.z, v.w, 16), v.w = __funnelshift_r(v.w, h, 16);
            }
          }
        }
        return v;
      };
      uint32_t top = 0;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 v = load(c);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
      }
      int ex = static_cast<int>(max(top & 0xFFFFu, top >> 16) >> 7) - 127;
      ex = max(-100, min(ex, 127));
      const float up = copysignf(__uint_as_float(static_cast<uint32_t>(12 - ex + 127) << 23), L.a.scale_log2);
      // (not zero, which would make a NaN of what is behind the prefix)
      f = fmaxf(fabsf(L.a.scale_log2) * __uint_as_float(static_cast<uint32_t>(ex - 12 + 127) << 23), 1e-37f);
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 v = load(c);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = half2_bits(__floats2half2_rn(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xFFFF0000u) * up));
        sts128(query + (c >> 3) * (kM * 128) + (((c & 7) ^ (tid & 7)) << 4), make_uint4(y[0], y[1], y[2], y[3]));
      }
    }
    async_fence();
    __syncwarp();
    if (lane == 0) w.arrive(kQueryFull + tile);
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int k = 0; k < 2 * p.count; ++k, ++mine) {
      const int h = k & 1;
      const int seen = p.len - p.t0 * kTile - k * kHalf;  // tokens of the half tile
      w.wait(kScoresFull + tile, mine);
      tc_fence_after();
      float x[2][32];
      tc_ld32(scores, x[0]);
      tc_ld32(scores + 32, x[1]);
      tc_wait_ld<32>(x[0]);
      tc_wait_ld<32>(x[1]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) w.arrive(kScoresRead + tile);
      if (seen < kHalf) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) x[i >> 5][i & 31] = i < seen ? x[i >> 5][i & 31] : -INFINITY;
      }
      uint32_t y[2][16];
      float sum;
      // First with the reference as it is: no weight is too large for fp16 if their sum is
      // not.  Else the reference becomes the row's maximum, and the sums so far follow.
#pragma unroll 1
      for (bool move = k == 0;; move = true) {
        if (move) {
          float top = x[0][0], top1 = x[1][0];
#pragma unroll
          for (int i = 1; i < 32; ++i) top = fmaxf(top, x[0][i]), top1 = fmaxf(top1, x[1][i]);
          top = fmaxf(top, top1);
          const float now = top == -INFINITY ? m : fmaxf(m, top * f), fall = ex2(m - now);
          if (k > 0) {
            w.wait(kOutFull + tile * 2 + (h ^ 1), (mine - 1) >> 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 8; ++c) {
              float o[8];
              uint32_t z[8];
              tc_ld8(out + c * 8, o);
              tc_wait_ld<8>(o);
#pragma unroll
              for (int i = 0; i < 8; ++i) z[i] = __float_as_uint(o[i] * fall);
              tc_st8(out + c * 8, z);
            }
            l *= fall;
          }
          m = now;
        }
        const uint32_t fb = __float_as_uint(f), rb = __float_as_uint(kFast - m);
        float part[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float a = 0.f, b = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float e0 = x[c][i], e1 = x[c][i + 1];
            fma_pair(e0, e1, make_uint4(fb, fb, rb, rb));
            e0 = ex2(e0), e1 = ex2(e1);
            add_pair(a, b, e0, e1);
            y[c][i >> 1] = half2_bits(__floats2half2_rn(e0, e1));
          }
          part[c] = a + b;
        }
        sum = part[0] + part[1];
        if (move || __all_sync(~0u, sum <= 65504.f)) break;
      }
      l += sum;
      // (the half before the last's weights have been read)
      w.wait(kOutFull + tile * 2 + h, (mine >> 1) ^ 1);
      tc_fence_after();
      tc_st16(weights + h * (kHalf / 2), y[0]);
      tc_st16(weights + h * (kHalf / 2) + 16, y[1]);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) w.arrive(kWeightsFull + tile * 2 + h);
    }
    // this part's sums
    w.wait(kOutFull + tile * 2, (mine - 2) >> 1);
    w.wait(kOutFull + tile * 2 + 1, (mine - 1) >> 1);
    tc_fence_after();
    const bool real = row < p.n_rows;
    const long long at = p.row0 + row + static_cast<long long>(blockIdx.x) * (2 * kM);
    constexpr float kUp = 1 << (kTop - kFast);  // (parts are kept 2^15 up)
    if (real) L.ml[at] = make_float2(m, w.dead() ? __int_as_float(0x7FC00000) : l * kUp);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      float x[32];
      tc_ld32(out + c * 32, x);
      tc_wait_ld<32>(x);
      if (real) {
        float4* o = reinterpret_cast<float4*>(L.o + at * D + c * 32);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = make_float4(x[4 * i] * kUp, x[4 * i + 1] * kUp, x[4 * i + 2] * kUp, x[4 * i + 3] * kUp);
      }
    }
    tc_fence_before();
  }
  if (w.dead() && lane == 0) atomicOr(L.a.status, 1 << SSD_ERR_CUDA);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) shared_tc_kernel(const __grid_constant__ SharedLaunch L) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long scan[kThreads], sums[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem) + 1023) & ~1023u;
  if (tid < kBars) {
    // how many warps (or commits) arrive
    int count = 1;
    if ((tid >= kKeysFull && tid < kKeysEmpty) || (tid >= kValuesFull && tid < kValuesEmpty) ||
        (tid >= kQueryFull && tid < kScoresFull) || (tid >= kScoresRead && tid < kOutFull))
      count = 4;
    if (tid >= kPartEmpty && tid < kPlaceFull) count = kReaders;
    if (tid >= kPlaceEmpty) count = 8;
    if ((tid >= kKeysEmpty && tid < kValuesFull) || (tid >= kValuesEmpty && tid < kQueryFull) || tid == kDone) count = 2;
    bar_init(base + tid * 8, count);
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + kTmemAt) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  tc_fence_before();
  GroupList list(L);
  list.build(scan, sums);
  tc_fence_after();
  Roles r = {L, base, lds32(base + kTmemAt), {}};
  r.w.bars = base;
  // 128 x (128 + 128 + 80 + 88 + 48) registers: within the 640 x 96 of the launch
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    weight_role<D>(r, warp >> 2, tid & 127);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    key_role<D>(r, tid & 127);
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    value_role<D>(r, tid & 127);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp < 18) matrix_role<D>(r, warp - 16, lane);
    else if (warp == 18) part_role(L, list, base, r.w, lane, kv_block_bytes(D));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(lds32(base + kTmemAt)));
  }
}

template <int D>
cudaError_t launch_dim(const SharedLaunch& L, cudaStream_t stream) {
  const cudaError_t e = allow_shared<shared_tc_kernel<D>>(Smem<D>::total);
  if (e != cudaSuccess) return e;
  shared_tc_kernel<D><<<L.teams, kThreads, Smem<D>::total, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_shared_tc(const SharedLaunch& L, int D, cudaStream_t stream) {
  return D == 64 ? launch_dim<64>(L, stream) : launch_dim<128>(L, stream);
}

}  // namespace ssdv
