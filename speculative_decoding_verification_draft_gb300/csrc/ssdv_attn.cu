// ssdv_attn.cu -- attention of a round's query tokens over the 4-bit cache.
//
// Query i of request b sits at position L_b + i and sees the positions
// [lo, hi): hi = L_b + i + 1 (its own key included), or L_b with past_only;
// lo = max(0, L_b + i + 1 - window) if there is a window, else 0.
//   out = sum_p exp(c q.k_p) v_p / sum_p exp(c q.k_p),  lse = log of that sum.
// A row that sees nothing has out = 0 and lse = -inf.
//
// One pass over the cache.  The rows of a request that share a kv head (query
// tokens x query heads of the group) meet each 64-token tile of keys and
// values in registers: S^T = K Q^T and O^T += V^T P^T on m16n8k16 fp16 matrix
// instructions with fp32 sums, the cache's side as the 16-wide operand, so that
// rows cost 8 at a time.  The tile's bytes come from shared memory, where bulk
// copies put whole 16-token blocks some tiles ahead; a thread's share of a
// fragment is contiguous in a block, so codes go from shared memory to
// fragments with one logic operation and one multiply-add per two values, and
// no value passes through shared memory a second time.  The values n s are
// exact in fp16.
//
// Queries enter as fp16 after a power of two per row (bf16: exact down to 2^-26
// of the row's largest element; fp32: as two fp16 parts).  Weights are rounded
// to fp16 for the second product (fp32 outputs: two parts), 2^15 at the largest
// of the row in the tile, so that they keep 11 bits down to 2^-29 of it; a tile
// with a smaller one, which real scores hardly hold, is passed over again for
// the octaves below.  Each tile's product is added to the row's fp32 sums with
// its own power of two, and maxima and sums of weights are in fp32.
//
// Work is split evenly whatever the lengths: every team of warps takes the same
// number of tiles of the list (request, kv head, tile).  Rows whose tiles are
// split between teams leave partial sums in the workspace, which a second
// kernel joins in the teams' order, so results do not depend on timing.
#include "ssdv_kv.cuh"

#include <algorithm>

namespace ssdv {

namespace {

constexpr int kTile = 64;        // tokens per tile: four blocks
constexpr int kBias = 15;        // weights are at most 2^kBias
constexpr int kBand = 29;        // octaves below that in which fp16 keeps 11 bits
constexpr int kBands = 5;        // passes a tile may take; weights below 2^-141 of its largest are dropped
constexpr float kSmallest = 6.103515625e-05f;  // 2^(kBias - kBand)
constexpr float kLowUp = 2048.f; // the second fp16 part of a weight is held this much up
constexpr int kMaxSms = 160;     // the workspace is sized for this many CTAs
constexpr int kSmem = 229000;    // dynamic shared memory, at most
constexpr int kMaxStages = 48;   // per CTA
constexpr int kHead = 1024;      // before the stages: 16 bytes of barriers and a flag per stage
constexpr int kWarps = 8;        // per CTA, one CTA per SM: up to 255 registers a thread

// Blocks lie 18 D + 32 bytes apart in shared memory: four consecutive blocks
// then start 32 bytes apart in the banks, which the value loads need.
__host__ __device__ constexpr int block_stride(int D) { return kv_block_bytes(D) + 32; }
__host__ __device__ constexpr int stage_bytes(int D) { return 4 * block_stride(D); }

// How the rows of a kv head are spread: up to nt n-tiles of 8 rows per warp, r
// warps (1, 2, 4 or 8) per team, all reading the same tile, rt passes over the
// cache; t teams per CTA with s stages each.
struct AttnShape {
  int nt, r, t, s, rt;
};

// Most n-tiles per warp that keep a warp's fragments in registers.
__host__ __device__ constexpr int max_nt(int D, bool f32) {
  return D == 64 ? (f32 ? 2 : 4) : D == 128 ? (f32 ? 2 : 3) : 1;
}

AttnShape attn_shape(int rows, int D, bool f32) {
  AttnShape p;
  const int n8 = (rows + 7) / 8, most = max_nt(D, f32);
  p.r = n8 <= most ? 1 : n8 <= 2 * most ? 2 : n8 <= 4 * most ? 4 : 8;
  p.nt = std::min((n8 + p.r - 1) / p.r, most);
  p.rt = (n8 + p.r * p.nt - 1) / (p.r * p.nt);
  p.t = kWarps / p.r;
  if (D == 256 && p.t == kWarps) p.t = 6;  // two stages each need it
  p.s = std::min({8, kMaxStages / p.t, (kSmem - kHead) / (p.t * stage_bytes(D))});
  return p;
}

struct AttnLaunch {
  KvAttnArgs a;
  AttnShape p;
  int per;          // query heads per kv head
  int rows;         // nq * per
  int rows_pass;    // r * nt * 8
  int4* desc;       // [teams]: request, head * rt + pass, parts, first slot
  float2* ml;       // [2 teams, rows_pass]: maximum and sum of a part
  float* o;         // [2 teams, rows_pass, D]
};

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
// False if the phase did not complete within the limit (some seconds).
__device__ __forceinline__ bool bar_wait(uint32_t bar, int parity) {
  for (int i = 0; i < (1 << 22); ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, int bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// ---- fragments ----

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
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
// ---- the list of work ----

// What a request's rows see together, and its tiles.
struct Span {
  int len, nq;     // query rows i < nq are real
  int lo, hi;      // positions some row sees
  int tile0, tiles;  // at least one tile, so that some team writes the outputs
  bool bad;
};
__device__ __forceinline__ Span find_span(const KvAttnArgs& a, int b) {
  Span s;
  s.len = a.kv_len[b];
  s.nq = a.n_q ? a.n_q[b] : a.nq;
  s.bad = s.len < 0 || s.nq < 0 || s.nq > a.nq ||
          static_cast<long long>(s.len) + (a.past_only ? 0 : s.nq) >
              static_cast<long long>(a.c.max_pages) * a.c.page_size;
  s.lo = s.hi = s.tile0 = 0;
  s.tiles = 1;
  if (s.bad || s.nq == 0) return s;
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
__device__ __forceinline__ int row_lo(const KvAttnArgs& a, int len, int i) {
  return a.window ? max(0, len + i + 1 - a.window) : 0;
}
__device__ __forceinline__ int row_hi(const KvAttnArgs& a, int len, int i) { return a.past_only ? len : len + i + 1; }

// A place in the list.
struct Place {
  int b, hr, tile;  // request, head * rt + pass, tile of the request's span
  Span s;
  __device__ __forceinline__ void next(const KvAttnArgs& a, int per_request) {
    if (++tile < s.tiles) return;
    tile = 0;
    if (++hr < per_request) return;
    hr = 0;
    if (++b < a.B) s = find_span(a, b);
  }
};

template <typename E>
__device__ __forceinline__ float query_at(const E* p, int d) {
  return static_cast<float>(p[d]);
}

// ---- the kernel ----

template <typename E, int D, int NT>
struct Rows {
  static constexpr bool kF32 = sizeof(E) == 4;
  static constexpr int kSteps = D / 16;  // k16 steps of a key row, and m16 tiles of a value row
  static constexpr int kParts = kF32 ? 2 : 1;
  uint32_t q[NT][kSteps][2 * kParts];
  float o[kSteps][NT][4];
  float f[NT][2];  // factor of a row's scores (log2 units)
  float m[NT][2], l[NT][2];
  // the lane's offsets in a tile: its first key row, that row's scales, its
  // values' block, its first value chunk there
  uint32_t key_at, scale_at, value_at, row_at;
  Bases bases;
  __device__ __forceinline__ void place(int lane) {
    const int r = lane >> 2, c = lane & 3;
    const uint32_t blk = (r >> 1) * block_stride(D);
    key_at = blk + (r & 1) * (D / 2) + (D == 64 ? c * 8 : c * 16) + (D == 256 ? (r & 1) * 64 : 0);
    scale_at = blk + kv_k_scales(D) + (D == 64 ? c * 16 + (r & 1) * 8 : c * 32 + (r & 1) * 16);
    value_at = c * block_stride(D);
    row_at = r * 16;
    bases = make_bases();
  }
};

// The element of a head that lane quarter c holds first in step s.
template <int D>
__device__ __forceinline__ int key_element(int c, int s) {
  if constexpr (D == 256) return (s >> 3) * 128 + c * 32 + (s & 7) * 4;
  return c * (D / 4) + s * 4;
}

template <typename E, int D, int NT>
__device__ __forceinline__ void load_queries(const AttnLaunch& L, Rows<E, D, NT>& w, int b, int h, int row0, int nrows,
                                             int lane) {
  using W = Rows<E, D, NT>;
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = row0 + nt * 8 + r;
    float x[W::kSteps][4];
    float top = 0.f;
    const bool real = row < nrows;
    const int i = real ? row / L.per : 0, g = real ? row % L.per : 0;
    const E* p = static_cast<const E*>(L.a.q) + b * L.a.qs[0] + i * L.a.qs[1] + (h * L.per + g) * L.a.qs[2];
#pragma unroll
    for (int s = 0; s < W::kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[s][e] = real ? query_at(p, key_element<D>(c, s) + e) : 0.f;
        top = fmaxf(top, fabsf(x[s][e]));
      }
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
    // the row's largest element to [2^12, 2^13)
    int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    ex = max(-100, min(ex, 127));
    // the scale's sign goes to the query, so that the largest product is the
    // largest score
    const float up = copysignf(__uint_as_float(static_cast<uint32_t>(12 - ex + 127) << 23), L.a.scale_log2);
    const float f = fabsf(L.a.scale_log2) * __uint_as_float(static_cast<uint32_t>(ex - 12 + 127) << 23);
    w.f[nt][0] = __shfl_sync(~0u, f, (2 * c) * 4);
    w.f[nt][1] = __shfl_sync(~0u, f, (2 * c + 1) * 4);
#pragma unroll
    for (int s = 0; s < W::kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float y0 = x[s][2 * e] * up, y1 = x[s][2 * e + 1] * up;
        const __half2 hi = __floats2half2_rn(y0, y1);
        w.q[nt][s][e] = half2_bits(hi);
        if constexpr (W::kF32) {
          const float2 back = __half22float2(hi);
          w.q[nt][s][2 + e] = half2_bits(__floats2half2_rn(y0 - back.x, y1 - back.y));
        }
      }
    w.m[nt][0] = w.m[nt][1] = -INFINITY;
    w.l[nt][0] = w.l[nt][1] = 0.f;
#pragma unroll
    for (int i2 = 0; i2 < W::kSteps; ++i2)
#pragma unroll
      for (int e = 0; e < 4; ++e) w.o[i2][nt][e] = 0.f;
  }
}

// One tile at `base` (shared memory) for the first NA n-tiles.  Token t of
// block k is row (k, t) of the fragments: S tile j holds tokens 4 j .. 4 j + 3
// of every block, fragment row r of it token 4 j + r % 2 of block r / 2 and row
// r + 8 the token two later.  `edge`: some row does not see some token.  Returns
// the further bands (bits) that a first pass, band 0, leaves to be done.
template <typename E, int D, int NT, int NA>
__device__ __forceinline__ uint32_t tile_step(const AttnLaunch& L, Rows<E, D, NT>& w, uint32_t base, int pos0, bool edge,
                                          const Span& sp, int row0, int lane, int band) {
  using W = Rows<E, D, NT>;
  constexpr int kStride = block_stride(D);
  const int r = lane >> 2, c = lane & 3;
  float s[4][NA][4];
  // scores
#pragma unroll
  for (int hh = 0; hh < (D == 256 ? 2 : 1); ++hh) {
    constexpr int kWords = D == 64 ? 2 : 4;
    const uint32_t blk = base + w.key_at;
    uint32_t sv[4];  // D = 64: bytes 2 j + y of 8; else bytes 2 y + g of word j (token y of two, group g of two)
    if constexpr (D == 64) {
      const uint2 x = lds64(base + w.scale_at);
      sv[0] = x.x, sv[1] = x.x >> 16, sv[2] = x.y, sv[3] = x.y >> 16;
    } else {
      const uint4 x = lds128(base + w.scale_at + hh * 128);
      sv[0] = x.x, sv[1] = x.y, sv[2] = x.z, sv[3] = x.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t wa[kWords], wb[kWords];
      if constexpr (D == 64) {
        const uint2 xa = lds64(blk + 4 * j * 32), xb = lds64(blk + (4 * j + 2) * 32);
        wa[0] = xa.x, wa[1] = xa.y, wb[0] = xb.x, wb[1] = xb.y;
      } else {
        const uint32_t at = hh ? blk + 64 - (r & 1) * 128 : blk;  // odd tokens' halves are exchanged
        const uint4 xa = lds128(at + 4 * j * (D / 2)), xb = lds128(at + (4 * j + 2) * (D / 2));
        wa[0] = xa.x, wa[1] = xa.y, wa[2] = xa.z, wa[3] = xa.w;
        wb[0] = xb.x, wb[1] = xb.y, wb[2] = xb.z, wb[3] = xb.w;
      }
#pragma unroll
      for (int g = 0; g < kWords / 2; ++g) {
        const uint32_t sa = __byte_perm(sv[j], 0, D == 64 ? 0x4040 : 0x4040 + 0x0101 * g) << 7;
        const uint32_t sb = __byte_perm(sv[j], 0, D == 64 ? 0x4141 : 0x4040 + 0x0101 * (2 + g)) << 7;
        const uint32_t a24 = mul2(sa, kMinus24), a264 = mul2(sa, kMinus264);
        const uint32_t b24 = mul2(sb, kMinus24), b264 = mul2(sb, kMinus264);
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // two words, two steps each
          const int word = 2 * g + (x >> 1), step = hh * 8 + 2 * word + (x & 1);
          const uint32_t ua = x & 1 ? __funnelshift_r(wa[word], wa[word], 8) : wa[word];
          const uint32_t ub = x & 1 ? __funnelshift_r(wb[word], wb[word], 8) : wb[word];
          const uint32_t a[4] = {fma2(pair_hi(ua, w.bases), sa, a24), fma2(pair_hi(ub, w.bases), sb, b24),
                                 fma2(pair_lo(ua, w.bases), sa, a264), fma2(pair_lo(ub, w.bases), sb, b264)};
#pragma unroll
          for (int nt = 0; nt < NA; ++nt) {
            if (step == 0) mma_first(s[j][nt], a, w.q[nt][step][0], w.q[nt][step][1]);
            else mma(s[j][nt], a, w.q[nt][step][0], w.q[nt][step][1]);
            if constexpr (W::kF32) mma(s[j][nt], a, w.q[nt][step][2], w.q[nt][step][3]);
          }
        }
      }
    }
  }
  // weights: 2^kBias at the tile's own maximum of the row
  uint32_t p[4][NA][2 * W::kParts];
  float grow[NA][2];  // factor of this pass's products
  uint32_t more = 0;
#pragma unroll
  for (int nt = 0; nt < NA; ++nt) {
    if (edge) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int i = (row0 + nt * 8 + 2 * c + x) / L.per;
        const int lo = row_lo(L.a, sp.len, i), hi = min(row_hi(L.a, sp.len, i), sp.hi);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int pos = pos0 + (r >> 1) * kKvBlock + 4 * j + (r & 1) + 2 * y;
            if (pos < lo || pos >= hi) s[j][nt][2 * y + x] = -INFINITY;
          }
      }
    }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) top[e & 1] = fmaxf(top[e & 1], s[j][nt][e]);
    float fall[2], ref[2], sum[2] = {0.f, 0.f};
    bool grown = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 4));
      top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 8));
      top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 16));
      if (top[x] != -INFINITY) top[x] *= w.f[nt][x];  // f >= 0
      const float m = fmaxf(w.m[nt][x], top[x]), zero = m == -INFINITY ? 0.f : m;
      grown |= m != w.m[nt][x];
      fall[x] = ex2(w.m[nt][x] - zero);  // the sums so far
      w.m[nt][x] = m;
      top[x] = top[x] == -INFINITY ? zero : top[x];
      grow[nt][x] = ex2(top[x] - zero - kBand * band);
      ref[x] = kBias - top[x];
    }
    float e[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) e[j][k] = ex2(fmaf(s[j][nt][k], w.f[nt][k & 1], ref[k & 1]));
    bool small = false;  // a weight below fp16's normal range
    if (edge) {
      // (a factor of zero makes no number of a masked score)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool seen = s[j][nt][k] != -INFINITY;
          e[j][k] = seen ? e[j][k] : 0.f;
          small |= seen && e[j][k] < kSmallest;
        }
    }
    __half2 least = __float2half2_rn(1.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 ha = __floats2half2_rn(e[j][0], e[j][1]), hb = __floats2half2_rn(e[j][2], e[j][3]);
      sum[0] += e[j][0] + e[j][2];
      sum[1] += e[j][1] + e[j][3];
      least = __hmin2(least, __hmin2(ha, hb));
      p[j][nt][0] = half2_bits(ha);
      p[j][nt][1] = half2_bits(hb);
    }
    // below 2^-14 fp16 keeps fewer bits: those weights go to a later band
    if (!edge) small = __low2float(least) < kSmallest || __high2float(least) < kSmallest;
    if (__any_sync(~0u, small) || band) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float u = fmaf(s[j][nt][k], w.f[nt][k & 1], ref[k & 1]);
          int at = u >= kBias - kBand ? 0 : min(kBands, static_cast<int>((kBias - u) * (1.f / kBand)));
          if (edge && s[j][nt][k] == -INFINITY) at = kBands;
          if (band == 0 && at > 0 && at < kBands) more |= 1u << at;
          e[j][k] = at == band ? ex2(u + kBand * band) : 0.f;
        }
        p[j][nt][0] = half2_bits(__floats2half2_rn(e[j][0], e[j][1]));
        p[j][nt][1] = half2_bits(__floats2half2_rn(e[j][2], e[j][3]));
      }
    }
    if (band == 0) {
      w.l[nt][0] = w.l[nt][0] * fall[0] + sum[0] * grow[nt][0];
      w.l[nt][1] = w.l[nt][1] * fall[1] + sum[1] * grow[nt][1];
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int i = 0; i < W::kSteps; ++i) {
          w.o[i][nt][0] *= fall[0], w.o[i][nt][2] *= fall[0];
          w.o[i][nt][1] *= fall[1], w.o[i][nt][3] *= fall[1];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (W::kF32) {
        const float2 fa = __half22float2(*reinterpret_cast<__half2*>(&p[j][nt][0]));
        const float2 fb = __half22float2(*reinterpret_cast<__half2*>(&p[j][nt][1]));
        p[j][nt][2] = transpose8(half2_bits(__floats2half2_rn((e[j][0] - fa.x) * kLowUp, (e[j][1] - fa.y) * kLowUp)));
        p[j][nt][3] = transpose8(half2_bits(__floats2half2_rn((e[j][2] - fb.x) * kLowUp, (e[j][3] - fb.y) * kLowUp)));
      }
      p[j][nt][0] = transpose8(p[j][nt][0]);
      p[j][nt][1] = transpose8(p[j][nt][1]);
    }
  }
  // values: lane quarter c takes block c, lane row r the elements r D/8 ..
  const uint32_t blk = base + w.value_at;
  constexpr int kGroups = D == 256 ? 2 : 1;
#pragma unroll
  for (int gg = 0; gg < kGroups; ++gg) {
    const int group = D == 64 ? r >> 1 : D == 128 ? r : 2 * r + gg;
    const uint4 vs = lds128(blk + kv_v_scales(D) + group * kKvBlock);
    uint32_t sc[4] = {vs.x, vs.y, vs.z, vs.w};
    uint32_t nans = 0;  // tokens of block c whose values of this group are NaN
    if (edge) {
      // what no row sees counts nothing whatever its bytes are; a NaN that some
      // row sees is taken out here and given to the rows that see it below
      const int first = pos0 + c * kKvBlock;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t byte = (sc[k >> 2] >> ((k & 3) * 8)) & 0xFFu;
        const bool seen = first + k >= sp.lo && first + k < sp.hi;
        if (seen && byte == kKvNanByte) nans |= 1u << k;
        if (!seen || byte == kKvNanByte) sc[k >> 2] &= ~(0xFFu << ((k & 3) * 8));
      }
    }
    uint32_t ss[4][4];  // per j: scales of its two token pairs and their offsets
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ss[j][0] = __byte_perm(sc[j], 0, 0x1404) >> 1;
      ss[j][1] = mul2(ss[j][0], kMinus24);
      ss[j][2] = __byte_perm(sc[j], 0, 0x3424) >> 1;
      ss[j][3] = mul2(ss[j][2], kMinus264);
    }
#pragma unroll
    for (int ii = 0; ii < W::kSteps / kGroups; ++ii) {
      const int i = gg * (W::kSteps / kGroups) + ii;
      const uint4 v = lds128(blk + kv_v_codes(D) + i * 128 + w.row_at);
      const uint32_t word[4] = {v.x, v.y, v.z, v.w};
      float t[NA][4];
      [[maybe_unused]] float t2[NA][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w0 = word[j >> 1], w1 = word[2 + (j >> 1)];
        const uint32_t u0 = j & 1 ? __funnelshift_r(w0, w0, 8) : w0;
        const uint32_t u1 = j & 1 ? __funnelshift_r(w1, w1, 8) : w1;
        const uint32_t a[4] = {fma2(pair_hi(u0, w.bases), ss[j][0], ss[j][1]), fma2(pair_hi(u1, w.bases), ss[j][0], ss[j][1]),
                               fma2(pair_lo(u0, w.bases), ss[j][2], ss[j][3]), fma2(pair_lo(u1, w.bases), ss[j][2], ss[j][3])};
#pragma unroll
        for (int nt = 0; nt < NA; ++nt) {
          if (j == 0) {
            mma_first(t[nt], a, p[j][nt][0], p[j][nt][1]);
            if constexpr (W::kF32) mma_first(t2[nt], a, p[j][nt][2], p[j][nt][3]);
          } else {
            mma(t[nt], a, p[j][nt][0], p[j][nt][1]);
            if constexpr (W::kF32) mma(t2[nt], a, p[j][nt][2], p[j][nt][3]);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NA; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (W::kF32) t[nt][e] = fmaf(t2[nt][e], 1.f / kLowUp, t[nt][e]);
          w.o[i][nt][e] = fmaf(t[nt][e], grow[nt][e & 1], w.o[i][nt][e]);
        }
    }
    if (edge && __any_sync(~0u, nans)) {
      for (int k = 0; k < 4; ++k) {
        const uint32_t there = __shfl_sync(~0u, nans, r * 4 + k);
        const int first = pos0 + k * kKvBlock;
#pragma unroll
        for (int nt = 0; nt < NA; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int i = (row0 + nt * 8 + 2 * c + x) / L.per;
            const int lo = row_lo(L.a, sp.len, i), hi = min(row_hi(L.a, sp.len, i), sp.hi);
            const int from = max(0, min(lo - first, 16)), to = max(0, min(hi - first, 16));
            if (there & ((1u << to) - 1u) & ~((1u << from) - 1u))
#pragma unroll
              for (int ii = 0; ii < W::kSteps / kGroups; ++ii) {
                w.o[gg * (W::kSteps / kGroups) + ii][nt][x] = __int_as_float(0x7FC00000);
                w.o[gg * (W::kSteps / kGroups) + ii][nt][2 + x] = __int_as_float(0x7FC00000);
              }
          }
      }
    }
  }
  return __any_sync(~0u, more) ? __reduce_or_sync(~0u, more) : 0u;
}

template <typename E, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, 1) kv_attention_kernel(const AttnLaunch L) {
  using W = Rows<E, D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long scan[kWarps * 32 + kWarps];
  const KvAttnArgs& a = L.a;
  const int R = L.p.r, T = L.p.t, S = L.p.s, RT = L.p.rt;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  const int team = warp / R;
  // the warp's place among the team's rows; rotated so that a short last group
  // does not always meet the same quarter of the SM
  const int part = (warp % R + team * R / 4) % R;
  const bool producer = warp % R == 0;
  const uint32_t base = smem_u32(smem);
  const uint32_t bars = base, data = base + kHead;
  volatile int* flags = reinterpret_cast<int*>(smem + 16 * kMaxStages);  // [T * S]: the stage lacks a bad page's block
  const auto full = [&](int st) { return bars + (team * S + st) * 16; };
  const auto empty = [&](int st) { return bars + (team * S + st) * 16 + 8; };
  const auto stage = [&](int st) { return data + (team * S + st) * stage_bytes(D); };
  if (tid < T * S) {
    bar_init(bars + tid * 16, 1);
    bar_init(bars + tid * 16 + 8, R);
    flags[tid] = 0;
  }
  // how many tiles there are, and where the teams begin
  const int chunk = (a.B + nthr - 1) / nthr;
  long long mine = 0;
  for (int b = tid * chunk; b < min(a.B, (tid + 1) * chunk); ++b) mine += find_span(a, b).tiles;
  long long x = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scan[kWarps * 32 + warp] = x;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();
  long long before = 0, total = 0;
  for (int v = 0; v < nthr / 32; ++v) {
    if (v < warp) before += scan[kWarps * 32 + v];
    total += scan[kWarps * 32 + v];
  }
  __syncthreads();
  scan[tid] = before + x - mine;
  __syncthreads();
  const int per_request = a.c.kv_heads * RT;
  const long long units = total * per_request;
  const long long teams = static_cast<long long>(gridDim.x) * T;
  const long long quota = (units + teams - 1) / teams;
  const long long me = static_cast<long long>(blockIdx.x) * T + team;
  const long long u_begin = me * quota, u_end = min(units, u_begin + quota);
  if (u_begin >= u_end) {
    if (producer && lane == 0) L.desc[me] = make_int4(0, 0, 0, 0);
    return;
  }
  Place at;
  long long u0;  // first unit of the request
  {
    int lo = 0, hi = nthr - 1;  // last thread whose requests begin at or before u_begin
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (scan[mid] * per_request <= u_begin && mid * chunk < a.B) lo = mid;
      else hi = mid - 1;
    }
    at.b = lo * chunk;
    u0 = scan[lo] * per_request;
    at.s = find_span(a, at.b);
    while (u0 + static_cast<long long>(at.s.tiles) * per_request <= u_begin) {
      u0 += static_cast<long long>(at.s.tiles) * per_request;
      at.s = find_span(a, ++at.b);
    }
    const long long k = u_begin - u0;
    at.hr = static_cast<int>(k / at.s.tiles);
    at.tile = static_cast<int>(k % at.s.tiles);
  }
  if (producer && lane == 0) {
    // the first team to begin inside a row's tiles has its parts joined
    const long long seg = u_begin - at.tile, prev = seg / quota;
    int4 d = make_int4(at.b, at.hr, 0, 0);
    if (at.tile > 0 && prev == me - 1) {
      d.z = static_cast<int>((seg + at.s.tiles - 1) / quota - prev + 1);
      d.w = static_cast<int>(2 * prev + (seg > prev * quota ? 1 : 0));
    }
    L.desc[me] = d;
  }

  // producing: lanes 0..3 of the team's first warp copy a block each
  const int n_tiles = static_cast<int>(u_end - u_begin);
  const int bpp = a.c.page_size / kKvBlock;
  Place pr = at;
  int issued = 0, page = -2;  // page of this lane's block of the next tile; -2: no block
  const auto fetch_page = [&]() {
    const int pos = (pr.s.tile0 + pr.tile) * kTile + (lane & 3) * kKvBlock;
    page = -2;
    if (pos < pr.s.hi && pos + kKvBlock > pr.s.lo)
      page = a.c.page_table[static_cast<long long>(pr.b) * a.c.max_pages + pos / kKvBlock / bpp];
  };
  const auto issue = [&]() -> bool {
    const int st = issued % S;
    if (R > 1 && issued >= S && !bar_wait(empty(st), (issued / S - 1) & 1)) return false;
    const int pb = (pr.s.tile0 + pr.tile) * (kTile / kKvBlock) + (lane & 3);
    const bool want = page != -2, ok = page >= 0 && page < a.c.n_pages;
    const uint32_t okm = __ballot_sync(~0u, ok) & 15u, badm = __ballot_sync(~0u, want && !ok) & 15u;
    if (lane == 0) {
      flags[team * S + st] = badm != 0;
      if (badm) atomicOr(a.status, 1 << SSD_ERR_PAGE);
      bar_expect(full(st), __popc(okm) * kv_block_bytes(D));
    }
    __syncwarp();
    if (lane < 4 && ok) {
      const long long k = (static_cast<long long>(page) * a.c.kv_heads + pr.hr / RT) * bpp + pb % bpp;
      bulk_copy(stage(st) + lane * block_stride(D), a.c.pages + k * kv_block_bytes(D), kv_block_bytes(D), full(st));
    }
    ++issued;
    if (issued < n_tiles) {
      pr.next(a, per_request);
      fetch_page();
    }
    return true;
  };
  bool alive = true;
  if (producer) {
    fetch_page();
    while (issued < n_tiles && issued < S) issue();
  }

  W w;
  w.place(lane);
  int done = 0;
  while (done < n_tiles && alive) {
    const int b = at.b, h = at.hr / RT, pass0 = (at.hr % RT) * L.rows_pass;
    const int first = at.tile, count = min(n_tiles - done, at.s.tiles - at.tile);
    const Span sp = at.s;
    const int nrows = sp.bad ? 0 : sp.nq * L.per;  // real rows of the request
    // the request's n-tiles, spread evenly over the team
    const int n8 = max(0, (min(nrows - pass0, L.rows_pass) + 7) / 8);
    const int row0 = pass0 + part * n8 / R * 8;
    const int own = (part + 1) * n8 / R - part * n8 / R;
    const int active = sp.hi > sp.lo ? own : 0;
    const int lo_last = row_lo(a, sp.len, sp.nq - 1), hi_first = row_hi(a, sp.len, 0);
    bool bad = sp.bad;
    load_queries<E, D, NT>(L, w, b, h, row0, nrows, lane);
    for (int k = 0; k < count; ++k, ++done) {
      const int st = done % S;
      if (!bar_wait(full(st), (done / S) & 1)) {
        alive = false;
        break;
      }
      bad |= flags[team * S + st] != 0;
      const int pos0 = (sp.tile0 + first + k) * kTile;
      const bool edge = pos0 < lo_last || pos0 + kTile > hi_first;
      for (uint32_t todo = active ? 1 : 0; todo;) {
        const int band = __ffs(todo) - 1;
        todo &= todo - 1;
        if (active == 1) todo |= tile_step<E, D, NT, 1>(L, w, stage(st), pos0, edge, sp, row0, lane, band);
        if constexpr (NT >= 2)
          if (active == 2) todo |= tile_step<E, D, NT, 2>(L, w, stage(st), pos0, edge, sp, row0, lane, band);
        if constexpr (NT >= 3)
          if (active == 3) todo |= tile_step<E, D, NT, 3>(L, w, stage(st), pos0, edge, sp, row0, lane, band);
        if constexpr (NT >= 4)
          if (active == 4) todo |= tile_step<E, D, NT, 4>(L, w, stage(st), pos0, edge, sp, row0, lane, band);
      }
      __syncwarp();
      if (R > 1 && lane == 0) bar_arrive(empty(st));
      // a team of several warps refills a tile late, when the others are done
      if (producer && issued < n_tiles && issued < done + 1 + S - (R > 1 ? 1 : 0) && !issue()) {
        alive = false;
        break;
      }
    }
    if (!alive) break;
    // this part's sums
    const int r = lane >> 2, c = lane & 3;
    const bool whole = first == 0 && count == sp.tiles;
    const long long slot = 2 * me + (first == 0 && done > count ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int xx = 0; xx < 2; ++xx) {
        float l = w.l[nt][xx];
        l += __shfl_xor_sync(~0u, l, 4);
        l += __shfl_xor_sync(~0u, l, 8);
        l += __shfl_xor_sync(~0u, l, 16);
        const int row = row0 + nt * 8 + 2 * c + xx;
        if (row >= nrows) l = 0.f;  // a padded query's row went along with its tile
        if (bad) l = __int_as_float(0x7FC00000);
        if (nt >= own || row >= L.rows) continue;
        if (whole) {
          const int i = row / L.per;
          const long long orow = (static_cast<long long>(b) * a.nq + i) * a.heads + h * L.per + row % L.per;
          const float inv = 1.f / l;
          float y[D / 8];
#pragma unroll
          for (int i2 = 0; i2 < W::kSteps; ++i2) {
            y[2 * i2] = l == 0.f ? 0.f : w.o[i2][nt][xx] * inv;
            y[2 * i2 + 1] = l == 0.f ? 0.f : w.o[i2][nt][2 + xx] * inv;
          }
          E* out = static_cast<E*>(a.out) + orow * D + r * (D / 8);
          if constexpr (W::kF32) {
#pragma unroll
            for (int v = 0; v < D / 32; ++v)
              reinterpret_cast<float4*>(out)[v] = make_float4(y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]);
          } else {
#pragma unroll
            for (int v = 0; v < D / 64; ++v) {
              uint32_t z[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 hh = __floats2bfloat162_rn(y[8 * v + 2 * e], y[8 * v + 2 * e + 1]);
                z[e] = *reinterpret_cast<const uint32_t*>(&hh);
              }
              reinterpret_cast<uint4*>(out)[v] = make_uint4(z[0], z[1], z[2], z[3]);
            }
          }
          if (a.lse && r == 0)
            a.lse[orow] = l == 0.f ? -INFINITY : (w.m[nt][xx] + (log2f(l) - kBias)) * 0.69314718055994531f;
        } else {
          const long long at_row = slot * L.rows_pass + (row - pass0);
          float* o = L.o + at_row * D + r * (D / 8);
#pragma unroll
          for (int v = 0; v < D / 32; ++v)
            reinterpret_cast<float4*>(o)[v] = make_float4(w.o[2 * v][nt][xx], w.o[2 * v][nt][2 + xx],
                                                          w.o[2 * v + 1][nt][xx], w.o[2 * v + 1][nt][2 + xx]);
          if (r == 0) L.ml[at_row] = make_float2(w.m[nt][xx], l);
        }
      }
    if (first == 0) {
      // rows past the request's own (all of them if its lengths are bad)
      if (sp.bad && at.hr == 0 && part == 0 && lane == 0) atomicOr(a.status, 1 << SSD_ERR_LENGTH);
      const float none = sp.bad ? __int_as_float(0x7FC00000) : 0.f;
      const int end = min(pass0 + L.rows_pass, L.rows);
      for (int row = pass0 + 8 * n8 + part; row < end; row += R) {
        const long long orow = (static_cast<long long>(b) * a.nq + row / L.per) * a.heads + h * L.per + row % L.per;
        for (int d = lane; d < D; d += 32) static_cast<E*>(a.out)[orow * D + d] = static_cast<E>(none);
        if (a.lse && lane == 0) a.lse[orow] = sp.bad ? none : -INFINITY;
      }
    }
    at.tile += count;
    if (at.tile == at.s.tiles) {
      at.tile = at.s.tiles - 1;
      at.next(a, per_request);
    }
  }
  if (!alive) {
    // a copy did not arrive in time: say so, and wait (with the same limit) for
    // the copies still in flight before the shared memory goes
    if (lane == 0) atomicOr(a.status, 1 << SSD_ERR_CUDA);
    if (producer)
      for (int k = done; k < issued; ++k)
        if (!bar_wait(full(k % S), (k / S) & 1)) break;
  }
}

// Joins the parts of one row's sums: one warp per row, teams in order.
template <typename E, int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const AttnLaunch L) {
  constexpr int kPer = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 d = L.desc[blockIdx.x];
  if (d.z == 0) return;
  const int lane = threadIdx.x & 31;
  const int RT = L.p.rt, local = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int row = (d.y % RT) * L.rows_pass + local;
  const int nrows = (L.a.n_q ? L.a.n_q[d.x] : L.a.nq) * L.per;
  if (local >= L.rows_pass || row >= min(L.rows, (nrows + 7) / 8 * 8)) return;
  // the first part's slot is d.w, the k-th after it is slot 0 of team d.w / 2 + k
  const auto slot = [&](int k) -> long long { return k == 0 ? d.w : 2LL * (d.w / 2 + k); };
  float m = -INFINITY;
  for (int k = lane; k < d.z; k += 32) m = fmaxf(m, L.ml[slot(k) * L.rows_pass + local].x);
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, y[kPer] = {};
#pragma unroll 4
  for (int k = 0; k < d.z; ++k) {
    const long long at = slot(k) * L.rows_pass + local;
    const float2 ml = L.ml[at];
    const float f = ex2(ml.x - ref);
    l += ml.y * f;
    const float* o = L.o + at * D + lane * kPer;
#pragma unroll
    for (int v = 0; v < kPer / 2; ++v) {
      const float2 z = reinterpret_cast<const float2*>(o)[v];
      // a part of weight zero counts nothing unless it holds a NaN
      y[2 * v] += z.x * f;
      y[2 * v + 1] += z.y * f;
    }
  }
  const int i = row / L.per, h = d.y / RT;
  const long long orow = (static_cast<long long>(d.x) * L.a.nq + i) * L.a.heads + h * L.per + row % L.per;
  const float inv = 1.f / l;
  E* out = static_cast<E*>(L.a.out) + orow * D + lane * kPer;
#pragma unroll
  for (int v = 0; v < kPer; ++v) out[v] = static_cast<E>(l == 0.f ? 0.f : y[v] * inv);
  if (L.a.lse && lane == 0)
    L.a.lse[orow] = l == 0.f ? -INFINITY : (ref + (log2f(l) - kBias)) * 0.69314718055994531f;
}

template <typename E, int D, int NT>
cudaError_t launch_nt(const AttnLaunch& L, int sms, cudaStream_t s) {
  const int smem = kHead + L.p.t * L.p.s * stage_bytes(D);
  cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<E, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kv_attention_kernel<E, D, NT><<<sms, L.p.t * L.p.r * 32, smem, s>>>(L);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms * L.p.t, (std::min(L.rows, L.rows_pass) + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<E, D>, L);
}

template <typename E, int D>
cudaError_t launch_dim(const AttnLaunch& L, int sms, cudaStream_t s) {
  constexpr int kMost = max_nt(D, sizeof(E) == 4);
  if constexpr (kMost >= 4)
    if (L.p.nt == 4) return launch_nt<E, D, 4>(L, sms, s);
  if constexpr (kMost >= 3)
    if (L.p.nt == 3) return launch_nt<E, D, 3>(L, sms, s);
  if constexpr (kMost >= 2)
    if (L.p.nt == 2) return launch_nt<E, D, 2>(L, sms, s);
  return launch_nt<E, D, 1>(L, sms, s);
}

struct WorkLayout {
  size_t desc, ml, o, total;
};
WorkLayout work_layout(const AttnShape& p, int D) {
  WorkLayout w;
  const size_t teams = static_cast<size_t>(kMaxSms) * p.t, rows = 2 * teams * p.r * p.nt * 8;
  w.desc = 0;
  w.ml = w.desc + teams * sizeof(int4);
  w.o = (w.ml + rows * sizeof(float2) + 255) / 256 * 256;
  w.total = w.o + rows * D * sizeof(float);
  return w;
}

}  // namespace

size_t kv_attention_work_bytes(int rows, int D) {
  return std::max(work_layout(attn_shape(rows, D, false), D).total, work_layout(attn_shape(rows, D, true), D).total);
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, int D, int esize, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  sms = std::min(sms, kMaxSms);
  AttnLaunch L;
  L.a = a;
  L.per = a.heads / a.c.kv_heads;
  L.rows = a.nq * L.per;
  L.p = attn_shape(L.rows, D, esize == 4);
  L.rows_pass = L.p.r * L.p.nt * 8;
  const WorkLayout w = work_layout(L.p, D);
  L.desc = reinterpret_cast<int4*>(a.work + w.desc);
  L.ml = reinterpret_cast<float2*>(a.work + w.ml);
  L.o = reinterpret_cast<float*>(a.work + w.o);
  if (esize == 2) {
    if (D == 64) return launch_dim<__nv_bfloat16, 64>(L, sms, stream);
    if (D == 128) return launch_dim<__nv_bfloat16, 128>(L, sms, stream);
    return launch_dim<__nv_bfloat16, 256>(L, sms, stream);
  }
  if (D == 64) return launch_dim<float, 64>(L, sms, stream);
  if (D == 128) return launch_dim<float, 128>(L, sms, stream);
  return launch_dim<float, 256>(L, sms, stream);
}

}  // namespace ssdv
