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
// with a smaller one is passed over again for the octaves below (128 requests, one
// query token: 82 us where no tile is, 176 with scores spread four times as far).
// Each tile's product is added to the row's fp32 sums with
// its own power of two, and maxima and sums of weights are in fp32.
//
// Measured: 128 requests of 301 to 6007 tokens, one query token, 4 query heads a
// kv head of 128 (8 kv heads): 80 us, 3.6 TB/s, bound by the latency of a tile's
// steps (two warps a scheduler issue 0.48 a cycle); twelve computing warps of 152
// registers in place of eight of 224: the same, and short requests slower.  32
// requests, 10 rows of 256: 60 us, 1.8 TB/s, also instruction fetches.
#include "ssdv_attn.cuh"

#include <algorithm>

namespace ssdv {

namespace {

constexpr int kTile = 64;        // tokens per tile: four blocks
constexpr int kBias = 15;        // weights are at most 2^kBias
constexpr float kLowUp = 2048.f; // the second fp16 part of a weight is held this much up
// More rows than this take ssdv_attn_tc.cu (bf16, 128 elements).  64 requests of 8
// kv heads, here against there: 16 rows 42 / 46 us for 500 tokens, 125 / 164 for
// 4000, 89 / 111 for 201 to 8003; 20 rows 52 / 51, 184 / 180 and 117 / 118; 40 rows
// 93 / 56 and 319 / 172 for 500 and 4000.
constexpr int kTcRows = 16;
constexpr int kSmem = 226000;    // dynamic shared memory, at most
constexpr int kWarps = 8;        // computing warps per CTA, one CTA per SM
constexpr int kThreads = 384;    // and four more, of which one keeps the copies going
// Beginning and ending a row's tiles costs as much as this many (64 requests of 201
// to 8003 tokens, 20 rows: 143 us at 0, 127 at 1, 117 at 2, 121 at 4).
constexpr int kPartTiles = 2;
constexpr int kMaxStages = 48;   // per CTA
constexpr int kHead = 1024;      // before the stages: 16 bytes of barriers and a flag per stage

// Blocks lie 18 D + 32 bytes apart in shared memory: four consecutive blocks
// then start 32 bytes apart in the banks, which the value loads need.
__host__ __device__ constexpr int block_stride(int D) { return kv_block_bytes(D) + 32; }
__host__ __device__ constexpr int stage_bytes(int D) { return 4 * block_stride(D); }

// Most n-tiles of 8 rows whose fragments stay in the registers of one warp, or
// of a pair of warps that halve the tile (p = 2: each takes half the tokens of
// the scores and half the elements of the values).
__host__ __device__ constexpr int max_nt(int D, bool f32, int p) {
  if (p == 1) return f32 ? (D == 256 ? 0 : 1) : D == 256 ? 1 : 2;
  return f32 ? (D == 64 ? 4 : D == 128 ? 3 : 2) : D == 256 ? 2 : 6;
}
// A pair keeps its queries in shared memory; a single warp has registers for them.
__host__ __device__ constexpr int query_bytes(int D, int nt, bool f32) { return nt * 8 * D * (f32 ? 4 : 2); }
// Two buffers of weights, then the maxima of both halves, the factors, the sums
// and the bands to come.
__host__ __device__ constexpr int exchange_bytes(int nt, bool f32) {
  return 2 * nt * 1024 * (f32 ? 2 : 1) + (2 * 2 + 1 + 2) * nt * 32 + 128;
}
__host__ __device__ constexpr int pair_bytes(int D, int nt, bool f32) {
  return query_bytes(D, nt, f32) + exchange_bytes(nt, f32);
}

AttnShape attn_shape(int rows, int D, bool f32) {
  AttnShape a;
  const int n8 = (rows + 7) / 8;
  a.tc = D == 128 && !f32 && rows > kTcRows;
  if (a.tc) {
    // passes of 32 to 64 rows, as even as they come
    a.rt = (rows + 63) / 64;
    a.nt = ((rows + a.rt - 1) / a.rt + 15) / 16 * 2;
    a.p = a.g = a.t = a.s = 1;
    return a;
  }
  a.p = n8 <= max_nt(D, f32, 1) ? 1 : 2;
  const int most = max_nt(D, f32, a.p);
  a.g = n8 <= most ? 1 : n8 <= 2 * most ? 2 : 4;
  a.nt = std::min((n8 + a.g - 1) / a.g, most);
  if (a.p == 2 && !f32 && D != 256) a.nt = std::max(a.nt, 3);
  a.rt = (n8 + a.g * a.nt - 1) / (a.g * a.nt);
  a.t = kWarps / (a.p * a.g);
  const int pairs = a.p == 2 ? a.g * pair_bytes(D, a.nt, f32) : 0;  // per team
  const auto stages = [&] { return ((kSmem - kHead) / a.t - pairs) / stage_bytes(D); };
  while (stages() < 2) --a.t;
  a.s = std::min({8, kMaxStages / a.t, stages()});
  return a;
}

// ---- fragments ----

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// ---- the kernel ----

// What a warp keeps of its rows: fragments of the queries (one warp alone),
// sums, maxima, and where its lanes read in a tile.
template <typename E, int D, int NT, int P>
struct Rows {
  static constexpr bool kF32 = sizeof(E) == 4;
  static constexpr int kSteps = D / 16;  // k16 steps of a key row, and m16 tiles of a value row
  static constexpr int kParts = kF32 ? 2 : 1;
  static constexpr int kJ = 4 / P;       // sets of 16 tokens that the warp scores
  static constexpr int kI = kSteps / P;  // value tiles that it sums
  uint32_t q[P == 1 ? NT : 1][P == 1 ? kSteps : 1][2 * kParts];
  float f[P == 1 ? NT : 1][2];  // factor of a row's scores (log2 units)
  float o[kI][NT][4];
  float m[NT][2], l[NT][2];
  // offsets in a tile: the lane's first key row, that row's scales, its values
  uint32_t key_at, scale_at, value_at;
  int pw;           // which of a pair
  uint32_t shared;  // a pair's queries and exchange
  const int2* span; // positions that each row sees
  Bases bases;

  static constexpr int kWeights = NT * 1024 * kParts;  // bytes of a tile's weights
  __device__ __forceinline__ uint32_t weights_at(int buf, int j, int nt, int lane) const {
    return shared + query_bytes(D, NT, kF32) + buf * kWeights + (j * NT + nt) * 256 * kParts + lane * 8 * kParts;
  }
  __device__ __forceinline__ uint32_t tops_at(int buf, int half) const {
    return shared + query_bytes(D, NT, kF32) + 2 * kWeights + (buf * 2 + half) * NT * 32;
  }
  __device__ __forceinline__ uint32_t factors_at() const { return tops_at(2, 0); }
  __device__ __forceinline__ uint32_t sums_at(int half) const { return tops_at(2, 1) + half * NT * 32; }
  __device__ __forceinline__ uint32_t more_at(int buf, int half) const { return sums_at(2) + (buf * 2 + half) * 4; }

  __device__ __forceinline__ void place(int lane, int pw_, uint32_t shared_, const int2* span_) {
    const int r = lane >> 2, c = lane & 3;
    const uint32_t blk = (r >> 1) * block_stride(D);
    pw = pw_;
    shared = shared_;
    span = span_;
    key_at = blk + (r & 1) * (D / 2) + (D == 64 ? c * 8 : c * 16) + pw * kJ * 4 * (D / 2);
    scale_at = blk + kv_k_scales(D) + (D == 64 ? c * 16 + (r & 1) * 8 + pw * 4 : c * 32 + (r & 1) * 16 + pw * 8);
    value_at = c * block_stride(D) + kv_v_codes(D) + pw * kI * 128 + r * 16;
    bases = make_bases();
  }
  __device__ __forceinline__ void query(int nt, int step, int lane, uint32_t (&b)[2 * kParts]) const {
    if constexpr (P == 1) {
#pragma unroll
      for (int x = 0; x < 2 * kParts; ++x) b[x] = q[nt][step][x];
    } else if constexpr (kF32) {
      const uint4 v = lds128(shared + (nt * kSteps + step) * 512 + lane * 16);
      b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
    } else {
      const uint2 v = lds64(shared + (nt * kSteps + step) * 256 + lane * 8);
      b[0] = v.x, b[1] = v.y;
    }
  }
  __device__ __forceinline__ void set_query(int nt, int step, int lane, const uint32_t (&b)[2 * kParts]) {
    if constexpr (P == 1) {
#pragma unroll
      for (int x = 0; x < 2 * kParts; ++x) q[nt][step][x] = b[x];
    } else if constexpr (kF32) {
      sts128(shared + (nt * kSteps + step) * 512 + lane * 16, make_uint4(b[0], b[1], b[2], b[3]));
    } else {
      sts64(shared + (nt * kSteps + step) * 256 + lane * 8, make_uint2(b[0], b[1]));
    }
  }
};

__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ float2 lds_f2(uint32_t p) {
  const uint2 v = lds64(p);
  return make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
}
__device__ __forceinline__ void sts_f2(uint32_t p, float x, float y) {
  sts64(p, make_uint2(__float_as_uint(x), __float_as_uint(y)));
}

// The element of a head that lane quarter c holds first in step s.
template <int D>
__device__ __forceinline__ int key_element(int c, int s) {
  if constexpr (D == 256) return (s >> 3) * 128 + c * 32 + (s & 7) * 4;
  return c * (D / 4) + s * 4;
}

template <typename E, int D, int NT, int P>
__device__ __forceinline__ void load_queries(const AttnLaunch& L, Rows<E, D, NT, P>& w, int b, int h, int row0, int nrows,
                                             const Span& sp, int2* span, int lane, int sync) {
  using W = Rows<E, D, NT, P>;
  const int r = lane >> 2, c = lane & 3;
  __syncwarp();  // the rows before are done with shared memory
  for (int k = lane; k < NT * 8; k += 32) {
    const int i = (row0 + k) / L.per;
    span[k] = make_int2(row_lo(L.a, sp.len, i), min(row_hi(L.a, sp.len, i), sp.hi));
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (P == 1 || nt % 2 == w.pw) {
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
          x[s][e] = real ? static_cast<float>(p[key_element<D>(c, s) + e]) : 0.f;
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
      const float f0 = __shfl_sync(~0u, f, (2 * c) * 4), f1 = __shfl_sync(~0u, f, (2 * c + 1) * 4);
      if constexpr (P == 1) {
        w.f[nt][0] = f0, w.f[nt][1] = f1;
      } else if (r == 0) {
        sts_f2(w.factors_at() + nt * 32 + c * 8, f0, f1);
      }
#pragma unroll
      for (int s = 0; s < W::kSteps; ++s) {
        uint32_t part[2 * W::kParts];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y0 = x[s][2 * e] * up, y1 = x[s][2 * e + 1] * up;
          const __half2 hi = __floats2half2_rn(y0, y1);
          part[e] = half2_bits(hi);
          if constexpr (W::kF32) {
            const float2 back = __half22float2(hi);
            part[2 + e] = half2_bits(__floats2half2_rn(y0 - back.x, y1 - back.y));
          }
        }
        w.set_query(nt, s, lane, part);
      }
    }
    w.m[nt][0] = w.m[nt][1] = -INFINITY;
    w.l[nt][0] = w.l[nt][1] = 0.f;
#pragma unroll
    for (int i2 = 0; i2 < W::kI; ++i2)
#pragma unroll
      for (int e = 0; e < 4; ++e) w.o[i2][nt][e] = 0.f;
  }
  __syncwarp();
  if constexpr (P == 2) pair_sync(sync);
}

// One tile at `base` (shared memory) for the first NA n-tiles.  Token t of
// block k is row (k, t) of the fragments: S tile j holds tokens 4 j .. 4 j + 3
// of every block, fragment row r of it token 4 j + r % 2 of block r / 2 and row
// r + 8 the token two later.  Of a pair, a warp scores two of the four j and
// hands the weights to the other, then sums half of the elements over all
// tokens; the one barrier per tile suffices because buffers alternate.
// `edge`: some row does not see some token.  Returns the further bands (bits)
// that a first pass, band 0, leaves to be done.
template <typename E, int D, int NT, int P, int NA>
__device__ __forceinline__ uint32_t tile_step(Rows<E, D, NT, P>& w, uint32_t base, int pos0, bool edge, int lo_seen,
                                              int hi_seen, int lane, int sync, int buf, int band) {
  using W = Rows<E, D, NT, P>;
  const int r = lane >> 2, c = lane & 3;
  float s[W::kJ][NA][4];
  // scores: kSets sets of 16 tokens go side by side, so that consecutive matrix
  // instructions do not wait on one another's sums
  constexpr int kSets = NA == 1 ? W::kJ : 2;
#pragma unroll
  for (int hh = 0; hh < (D == 256 ? 2 : 1); ++hh) {
    constexpr int kWords = D == 64 ? 2 : 4;
    // D = 256: odd tokens' halves are exchanged
    const uint32_t blk = base + w.key_at + (D == 256 ? (hh ^ (r & 1)) * 64 : 0);
    uint32_t sv[4];  // D = 64: bytes y of word j; else bytes 2 y + g (token y of two, group g of two)
    if constexpr (D == 64 && P == 1) {
      const uint2 x = lds64(base + w.scale_at);
      sv[0] = x.x, sv[1] = x.x >> 16, sv[2] = x.y, sv[3] = x.y >> 16;
    } else if constexpr (D == 64) {
      sv[0] = lds32(base + w.scale_at), sv[1] = sv[0] >> 16;
    } else if constexpr (P == 1) {
      const uint4 x = lds128(base + w.scale_at + hh * 128);
      sv[0] = x.x, sv[1] = x.y, sv[2] = x.z, sv[3] = x.w;
    } else {
      const uint2 x = lds64(base + w.scale_at + hh * 128);
      sv[0] = x.x, sv[1] = x.y;
    }
#pragma unroll
    for (int j0 = 0; j0 < W::kJ; j0 += kSets) {
      uint32_t wa[kSets][kWords], wb[kSets][kWords];
#pragma unroll
      for (int j = 0; j < kSets; ++j) {
        const uint32_t at = blk + 4 * (j0 + j) * (D / 2);
        if constexpr (D == 64) {
          const uint2 xa = lds64(at), xb = lds64(at + 2 * (D / 2));
          wa[j][0] = xa.x, wa[j][1] = xa.y, wb[j][0] = xb.x, wb[j][1] = xb.y;
        } else {
          const uint4 xa = lds128(at), xb = lds128(at + 2 * (D / 2));
          wa[j][0] = xa.x, wa[j][1] = xa.y, wa[j][2] = xa.z, wa[j][3] = xa.w;
          wb[j][0] = xb.x, wb[j][1] = xb.y, wb[j][2] = xb.z, wb[j][3] = xb.w;
        }
      }
#pragma unroll
      for (int g = 0; g < kWords / 2; ++g) {
        uint32_t sc[kSets][6];
#pragma unroll
        for (int j = 0; j < kSets; ++j) {
          sc[j][0] = __byte_perm(sv[j0 + j], 0, D == 64 ? 0x4040 : 0x4040 + 0x0101 * g) << 7;
          sc[j][1] = __byte_perm(sv[j0 + j], 0, D == 64 ? 0x4141 : 0x4040 + 0x0101 * (2 + g)) << 7;
          sc[j][2] = mul2(sc[j][0], kMinus24), sc[j][3] = mul2(sc[j][0], kMinus264);
          sc[j][4] = mul2(sc[j][1], kMinus24), sc[j][5] = mul2(sc[j][1], kMinus264);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // two words, two steps each
          const int word = 2 * g + (x >> 1), step = hh * 8 + 2 * word + (x & 1);
          uint32_t q[NA][2 * W::kParts];
#pragma unroll
          for (int nt = 0; nt < NA; ++nt) w.query(nt, step, lane, q[nt]);
#pragma unroll
          for (int j = 0; j < kSets; ++j) {
            const uint32_t ua = x & 1 ? __funnelshift_r(wa[j][word], wa[j][word], 8) : wa[j][word];
            const uint32_t ub = x & 1 ? __funnelshift_r(wb[j][word], wb[j][word], 8) : wb[j][word];
            const uint32_t a[4] = {
                fma2(pair_hi(ua, w.bases), sc[j][0], sc[j][2]), fma2(pair_hi(ub, w.bases), sc[j][1], sc[j][4]),
                fma2(pair_lo(ua, w.bases), sc[j][0], sc[j][3]), fma2(pair_lo(ub, w.bases), sc[j][1], sc[j][5])};
#pragma unroll
            for (int nt = 0; nt < NA; ++nt) {
              if (step == 0) mma_first(s[j0 + j][nt], a, q[nt][0], q[nt][1]);
              else mma(s[j0 + j][nt], a, q[nt][0], q[nt][1]);
              if constexpr (W::kF32) mma(s[j0 + j][nt], a, q[nt][2], q[nt][3]);
            }
          }
        }
      }
    }
  }
  // weights: 2^kBias at the maximum of the row in the warp's tokens
  uint32_t p[4][NA][2 * W::kParts];
  float grow[NA][P][2];  // factors of this pass's products
  float sum[NA][2];
  uint32_t more = 0;
#pragma unroll
  for (int nt = 0; nt < NA; ++nt) {
    float f[2];
    if constexpr (P == 1) {
      f[0] = w.f[nt][0], f[1] = w.f[nt][1];
    } else {
      const float2 x = lds_f2(w.factors_at() + nt * 32 + c * 8);
      f[0] = x.x, f[1] = x.y;
    }
    if (edge) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int2 seen = w.span[nt * 8 + 2 * c + x];
#pragma unroll
        for (int j = 0; j < W::kJ; ++j)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int pos = pos0 + (r >> 1) * kKvBlock + 4 * (w.pw * W::kJ + j) + (r & 1) + 2 * y;
            if (pos < seen.x || pos >= seen.y) s[j][nt][2 * y + x] = -INFINITY;
          }
      }
    }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < W::kJ; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) top[k & 1] = fmaxf(top[k & 1], s[j][nt][k]);
    float ref[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 4));
      top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 8));
      top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 16));
      if (top[x] != -INFINITY) top[x] *= f[x];  // f >= 0
      ref[x] = kBias - (top[x] == -INFINITY ? 0.f : top[x]);
    }
    float e[W::kJ][4];
#pragma unroll
    for (int j = 0; j < W::kJ; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) e[j][k] = ex2(fmaf(s[j][nt][k], f[k & 1], ref[k & 1]));
    bool small = false;  // a weight below fp16's normal range
    if (edge) {
      // (a factor of zero makes no number of a masked score)
#pragma unroll
      for (int j = 0; j < W::kJ; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool seen = s[j][nt][k] != -INFINITY;
          e[j][k] = seen ? e[j][k] : 0.f;
          small |= seen && e[j][k] < kSmallest;
        }
    }
    sum[nt][0] = sum[nt][1] = 0.f;
    __half2 least = __float2half2_rn(1.f);
    uint32_t ph[W::kJ][2];
#pragma unroll
    for (int j = 0; j < W::kJ; ++j) {
      const __half2 ha = __floats2half2_rn(e[j][0], e[j][1]), hb = __floats2half2_rn(e[j][2], e[j][3]);
      sum[nt][0] += e[j][0] + e[j][2];
      sum[nt][1] += e[j][1] + e[j][3];
      least = __hmin2(least, __hmin2(ha, hb));
      ph[j][0] = half2_bits(ha);
      ph[j][1] = half2_bits(hb);
    }
    // below 2^-14 fp16 keeps fewer bits: those weights go to a later band
    if (!edge) small = __low2float(least) < kSmallest || __high2float(least) < kSmallest;
    if (__any_sync(~0u, small) || band) {
#pragma unroll
      for (int j = 0; j < W::kJ; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float u = fmaf(s[j][nt][k], f[k & 1], ref[k & 1]);
          int at = u >= kBias - kBand ? 0 : min(kBands, static_cast<int>((kBias - u) * (1.f / kBand)));
          if (edge && s[j][nt][k] == -INFINITY) at = kBands;
          if (band == 0 && at > 0 && at < kBands) more |= 1u << at;
          e[j][k] = at == band ? ex2(u + kBand * band) : 0.f;
        }
        ph[j][0] = half2_bits(__floats2half2_rn(e[j][0], e[j][1]));
        ph[j][1] = half2_bits(__floats2half2_rn(e[j][2], e[j][3]));
      }
    }
#pragma unroll
    for (int j = 0; j < W::kJ; ++j) {
      uint32_t y[2 * W::kParts];
      y[0] = transpose8(ph[j][0]);
      y[1] = transpose8(ph[j][1]);
      if constexpr (W::kF32) {
        const float2 fa = __half22float2(*reinterpret_cast<__half2*>(&ph[j][0]));
        const float2 fb = __half22float2(*reinterpret_cast<__half2*>(&ph[j][1]));
        y[2] = transpose8(half2_bits(__floats2half2_rn((e[j][0] - fa.x) * kLowUp, (e[j][1] - fa.y) * kLowUp)));
        y[3] = transpose8(half2_bits(__floats2half2_rn((e[j][2] - fb.x) * kLowUp, (e[j][3] - fb.y) * kLowUp)));
      }
      if constexpr (P == 1) {
#pragma unroll
        for (int x = 0; x < 2 * W::kParts; ++x) p[j][nt][x] = y[x];
      } else {
        const uint32_t at = w.weights_at(buf, w.pw * W::kJ + j, nt, lane);
        if constexpr (W::kF32) sts128(at, make_uint4(y[0], y[1], y[2], y[3]));
        else sts64(at, make_uint2(y[0], y[1]));
      }
    }
    if constexpr (P == 1) {
      grow[nt][0][0] = top[0], grow[nt][0][1] = top[1];
    } else if (r == 0) {
      sts_f2(w.tops_at(buf, w.pw) + nt * 32 + c * 8, top[0], top[1]);
    }
  }
  more = __any_sync(~0u, more) ? __reduce_or_sync(~0u, more) : 0u;
  if constexpr (P == 2) {
    if (lane == 0) sts32(w.more_at(buf, w.pw), more);
    pair_sync(sync);
    more = lds32(w.more_at(buf, 0)) | lds32(w.more_at(buf, 1));
#pragma unroll
    for (int nt = 0; nt < NA; ++nt) {
#pragma unroll
      for (int h = 0; h < P; ++h) {
        const float2 x = lds_f2(w.tops_at(buf, h) + nt * 32 + c * 8);
        grow[nt][h][0] = x.x, grow[nt][h][1] = x.y;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = w.weights_at(buf, j, nt, lane);
        if constexpr (W::kF32) {
          const uint4 x = lds128(at);
          p[j][nt][0] = x.x, p[j][nt][1] = x.y, p[j][nt][2] = x.z, p[j][nt][3] = x.w;
        } else {
          const uint2 x = lds64(at);
          p[j][nt][0] = x.x, p[j][nt][1] = x.y;
        }
      }
    }
  }
  // the row's maximum so far, and what that makes of the sums so far and of
  // this tile's
#pragma unroll
  for (int nt = 0; nt < NA; ++nt) {
    float fall[2];
    bool grown = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float m = w.m[nt][x];
#pragma unroll
      for (int h = 0; h < P; ++h) m = fmaxf(m, grow[nt][h][x]);
      const float zero = m == -INFINITY ? 0.f : m;
      grown |= m != w.m[nt][x];
      fall[x] = ex2(w.m[nt][x] - zero);
      w.m[nt][x] = m;
#pragma unroll
      for (int h = 0; h < P; ++h) grow[nt][h][x] = ex2(grow[nt][h][x] - zero - kBand * band);
    }
    if (band == 0) {
      const float g0 = P == 2 && w.pw ? grow[nt][P - 1][0] : grow[nt][0][0];
      const float g1 = P == 2 && w.pw ? grow[nt][P - 1][1] : grow[nt][0][1];
      w.l[nt][0] = w.l[nt][0] * fall[0] + sum[nt][0] * g0;
      w.l[nt][1] = w.l[nt][1] * fall[1] + sum[nt][1] * g1;
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int i = 0; i < W::kI; ++i) {
          w.o[i][nt][0] *= fall[0], w.o[i][nt][2] *= fall[0];
          w.o[i][nt][1] *= fall[1], w.o[i][nt][3] *= fall[1];
        }
      }
    }
  }
  // values: lane quarter c takes block c, lane row r the elements r D/8 ..
  constexpr int kGroups = D == 256 && P == 1 ? 2 : 1;
#pragma unroll
  for (int gg = 0; gg < kGroups; ++gg) {
    const int group = D == 64 ? r >> 1 : D == 128 ? r : 2 * r + (P == 1 ? gg : w.pw);
    const uint4 vs = lds128(base + c * block_stride(D) + kv_v_scales(D) + group * kKvBlock);
    uint32_t sc[4] = {vs.x, vs.y, vs.z, vs.w};
    uint32_t nans = 0;  // tokens of block c whose values of this group are NaN
    if (edge) {
      // what no row sees counts nothing whatever its bytes are; a NaN that some
      // row sees is taken out here and given to the rows that see it below
      const int first = pos0 + c * kKvBlock;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t byte = (sc[k >> 2] >> ((k & 3) * 8)) & 0xFFu;
        const bool seen = first + k >= lo_seen && first + k < hi_seen;
        if (seen && byte == kKvNanByte) nans |= 1u << k;
        if (!seen || byte == kKvNanByte) sc[k >> 2] &= ~(0xFFu << ((k & 3) * 8));
      }
    }
    uint32_t ss[4][4];  // per j: scales of its two token pairs and their offsets
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ss[j][0] = __byte_perm(sc[j], 0, 0x4140) << 7;
      ss[j][1] = mul2(ss[j][0], kMinus24);
      ss[j][2] = __byte_perm(sc[j], 0, 0x4342) << 7;
      ss[j][3] = mul2(ss[j][2], kMinus264);
    }
    constexpr int kMost = W::kI / kGroups, kSide = NA == 1 ? (kMost < 4 ? kMost : 4) : NA == 2 ? 2 : 1;
#pragma unroll
    for (int ii = 0; ii < kMost; ii += kSide) {
      const int i0 = gg * kMost + ii;
      uint32_t word[kSide][4];
#pragma unroll
      for (int i = 0; i < kSide; ++i) {
        const uint4 v = lds128(base + w.value_at + (i0 + i) * 128);
        word[i][0] = v.x, word[i][1] = v.y, word[i][2] = v.z, word[i][3] = v.w;
      }
#pragma unroll
      for (int h = 0; h < P; ++h) {
        float t[kSide][NA][4];
        [[maybe_unused]] float t2[kSide][NA][4];
#pragma unroll
        for (int jj = 0; jj < W::kJ; ++jj)
#pragma unroll
          for (int i = 0; i < kSide; ++i) {
            const int j = h * W::kJ + jj;
            const uint32_t w0 = word[i][j >> 1], w1 = word[i][2 + (j >> 1)];
            const uint32_t u0 = j & 1 ? __funnelshift_r(w0, w0, 8) : w0;
            const uint32_t u1 = j & 1 ? __funnelshift_r(w1, w1, 8) : w1;
            const uint32_t a[4] = {
                fma2(pair_hi(u0, w.bases), ss[j][0], ss[j][1]), fma2(pair_hi(u1, w.bases), ss[j][0], ss[j][1]),
                fma2(pair_lo(u0, w.bases), ss[j][2], ss[j][3]), fma2(pair_lo(u1, w.bases), ss[j][2], ss[j][3])};
#pragma unroll
            for (int nt = 0; nt < NA; ++nt) {
              if (jj == 0) {
                mma_first(t[i][nt], a, p[j][nt][0], p[j][nt][1]);
                if constexpr (W::kF32) mma_first(t2[i][nt], a, p[j][nt][2], p[j][nt][3]);
              } else {
                mma(t[i][nt], a, p[j][nt][0], p[j][nt][1]);
                if constexpr (W::kF32) mma(t2[i][nt], a, p[j][nt][2], p[j][nt][3]);
              }
            }
          }
#pragma unroll
        for (int i = 0; i < kSide; ++i)
#pragma unroll
          for (int nt = 0; nt < NA; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (W::kF32) t[i][nt][k] = fmaf(t2[i][nt][k], 1.f / kLowUp, t[i][nt][k]);
              w.o[i0 + i][nt][k] = fmaf(t[i][nt][k], grow[nt][h][k & 1], w.o[i0 + i][nt][k]);
            }
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
            const int2 seen = w.span[nt * 8 + 2 * c + x];
            const int from = max(0, min(seen.x - first, 16)), to = max(0, min(seen.y - first, 16));
            if (there & ((1u << to) - 1u) & ~((1u << from) - 1u))
#pragma unroll
              for (int ii = 0; ii < kMost; ++ii) {
                w.o[gg * kMost + ii][nt][x] = __int_as_float(0x7FC00000);
                w.o[gg * kMost + ii][nt][2 + x] = __int_as_float(0x7FC00000);
              }
          }
      }
    }
  }
  return more;
}

// Keeps the copies of all teams going: four lanes per team, a block each.
template <int D>
__device__ __forceinline__ void produce(const AttnLaunch& L, const List<kTile>& list, uint32_t bars, uint32_t data,
                                        volatile int* flags, int lane) {
  const KvAttnArgs& a = L.a;
  const int S = L.p.s, RT = L.p.rt, team = lane >> 2;
  const int bpp = a.c.page_size / kKvBlock;
  const long long head_bytes = static_cast<long long>(bpp) * kv_block_bytes(D), page_bytes = head_bytes * a.c.kv_heads;
  typename List<kTile>::Share share = {};
  if (team < L.p.t) share = list.share(a, static_cast<long long>(blockIdx.x) * L.p.t + team);
  int left = share.count;
  Place<kTile> pr = share.at;
  int put = 0, phase = 1;     // empty stages at first
  int sub = 0, column = 0;    // this lane's block: of which page column, and where in the page
  int page = 0;
  bool want = false;          // the next tile has this lane's block
  const auto locate = [&]() {
    const int pb = (pr.s.tile0 + pr.tile) * (kTile / kKvBlock) + (lane & 3);
    column = pb / bpp;
    sub = pb % bpp;
  };
  const auto fetch_page = [&]() {
    const int pos = (pr.s.tile0 + pr.tile) * kTile + (lane & 3) * kKvBlock;
    want = pos < pr.s.hi && pos + kKvBlock > pr.s.lo;
    if (want) page = a.c.page_table[static_cast<long long>(pr.b) * a.c.max_pages + column];
  };
  if (left) {
    locate();
    fetch_page();
  }
  __syncwarp();
  long long idle = 0;
  while (__any_sync(~0u, left > 0)) {
    const uint32_t bar = bars + (team * S + put) * 16;
    bool ready = left > 0 && (lane & 3) == 0 && bar_test(bar + 8, phase);
    ready = __shfl_sync(~0u, ready, lane & 28);
    if (!__any_sync(~0u, ready)) {
      if (late(idle)) break;
      continue;
    }
    idle = 0;
    const bool ok = ready && want && page >= 0 && page < a.c.n_pages;
    const uint32_t okm = __ballot_sync(~0u, ok) >> (lane & 28) & 15u;
    const uint32_t bad = __ballot_sync(~0u, ready && want && !ok) >> (lane & 28) & 15u;
    if (ready && (lane & 3) == 0) {
      flags[team * S + put] = bad != 0;
      if (bad) atomicOr(a.status, 1 << SSD_ERR_PAGE);
      bar_expect(bar, __popc(okm) * kv_block_bytes(D));
    }
    __syncwarp();
    if (ok)
      bulk_copy(data + (team * S + put) * stage_bytes(D) + (lane & 3) * block_stride(D),
                a.c.pages + page * page_bytes + pr.hr / RT * head_bytes + static_cast<long long>(sub) * kv_block_bytes(D),
                kv_block_bytes(D), bar);
    if (ready) {
      if (++put == S) put = 0, phase ^= 1;
      if (--left) {
        pr.next(a, list.per_request);
        if (pr.tile == 0 || bpp < 4) {
          locate();
        } else if ((sub += 4) >= bpp) {
          sub -= bpp;
          ++column;
        }
        fetch_page();
      }
    }
    __syncwarp();
  }
  if (left > 0 && (lane & 3) == 0) atomicOr(a.status, 1 << SSD_ERR_CUDA);
}

template <typename E, int D, int NT, int P>
__device__ __forceinline__ void consume(const AttnLaunch& L, const List<kTile>& list, uint32_t bars, uint32_t data,
                                        volatile int* flags, int2* spans, int warp, int lane) {
  using W = Rows<E, D, NT, P>;
  const KvAttnArgs& a = L.a;
  const int S = L.p.s, RT = L.p.rt, G = L.p.g, T = L.p.t;
  const int team = warp / (P * G), group = warp / P % G, pw = warp % P;
  const int sync = 1 + warp / P;  // the pair's barrier
  const long long me = static_cast<long long>(blockIdx.x) * T + team;
  const typename List<kTile>::Share share = list.share(a, me);
  const bool first_warp = group == 0 && pw == 0;
  if (first_warp && lane == 0) L.desc[me] = list.parts(share, me);
  if (share.count == 0) return;
  Place<kTile> at = share.at;
  W w;
  w.place(lane, pw,
          P == 2 ? data + T * S * stage_bytes(D) + (warp / P) * pair_bytes(D, NT, W::kF32) : 0u, spans);
  const int n_tiles = share.count;
  int take = 0, phase = 0, buf = 0;
  int done = 0;
  bool dead = false;  // a copy did not arrive in time: go through the motions, without waiting
  while (done < n_tiles) {
    const int b = at.b, h = at.hr / RT, pass0 = (at.hr % RT) * L.rows_pass;
    const int first = at.tile, count = min(n_tiles - done, at.s.tiles - at.tile);
    const Span sp = at.s;
    const int nrows = sp.bad ? 0 : sp.nq * L.per;  // real rows of the request
    // the request's n-tiles, spread evenly over the team's groups
    const int n8 = max(0, (min(nrows - pass0, L.rows_pass) + 7) / 8);
    const int row0 = pass0 + group * n8 / G * 8;
    const int own = (group + 1) * n8 / G - group * n8 / G;
    const int active = sp.hi > sp.lo ? own : 0;
    const int lo_last = row_lo(a, sp.len, sp.nq - 1), hi_first = row_hi(a, sp.len, 0);
    bool bad = sp.bad;
    load_queries<E, D, NT, P>(L, w, b, h, row0, nrows, sp, spans, lane, sync);
    for (int k = 0; k < count; ++k, ++done) {
      const uint32_t bar = bars + (team * S + take) * 16;
      if (!dead && !bar_wait(bar, phase)) dead = true;
      bad |= flags[team * S + take] != 0;
      const uint32_t tile = data + (team * S + take) * stage_bytes(D);
      const int pos0 = (sp.tile0 + first + k) * kTile;
      const bool edge = pos0 < lo_last || pos0 + kTile > hi_first;
      for (uint32_t todo = active ? 1 : 0; todo;) {
        const int band = __ffs(todo) - 1;
        todo &= todo - 1;
        constexpr int kHalf = (NT + 1) / 2;
        if (kHalf < NT && active <= kHalf)
          todo |= tile_step<E, D, NT, P, kHalf>(w, tile, pos0, edge, sp.lo, sp.hi, lane, sync, buf, band);
        else
          todo |= tile_step<E, D, NT, P, NT>(w, tile, pos0, edge, sp.lo, sp.hi, lane, sync, buf, band);
        buf ^= 1;
      }
      __syncwarp();
      if (lane == 0) bar_arrive(bar + 8);
      if (++take == S) take = 0, phase ^= 1;
    }
    bad |= dead;
    // this part's sums
    const int r = lane >> 2, c = lane & 3;
    const bool whole = first == 0 && count == sp.tiles;
    const long long slot = 2 * me + (first == 0 && done > count ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        w.l[nt][x] += __shfl_xor_sync(~0u, w.l[nt][x], 4);
        w.l[nt][x] += __shfl_xor_sync(~0u, w.l[nt][x], 8);
        w.l[nt][x] += __shfl_xor_sync(~0u, w.l[nt][x], 16);
      }
    if constexpr (P == 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (r == 0) sts_f2(w.sums_at(pw) + nt * 32 + c * 8, w.l[nt][0], w.l[nt][1]);
      pair_sync(sync);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 l0 = lds_f2(w.sums_at(0) + nt * 32 + c * 8), l1 = lds_f2(w.sums_at(1) + nt * 32 + c * 8);
        w.l[nt][0] = l0.x + l1.x;
        w.l[nt][1] = l0.y + l1.y;
      }
      pair_sync(sync);
    }
    constexpr int kOwn = 2 * W::kI;  // elements of a row that a lane holds
    const int d0 = r * (D / 8) + pw * kOwn;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = row0 + nt * 8 + 2 * c + x;
        if (nt >= own || row >= nrows) continue;  // (a padded query's row went along with its tile)
        float l = w.l[nt][x];
        if (bad) l = __int_as_float(0x7FC00000);
        if (whole) {
          const int i = row / L.per;
          const long long orow = (static_cast<long long>(b) * a.nq + i) * a.heads + h * L.per + row % L.per;
          const float inv = 1.f / l;
          E* out = static_cast<E*>(a.out) + orow * D + d0;
#pragma unroll
          for (int v = 0; v < kOwn / 4; ++v) {
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = l == 0.f ? 0.f : w.o[2 * v + (k >> 1)][nt][x + 2 * (k & 1)] * inv;
            if constexpr (W::kF32) {
              reinterpret_cast<float4*>(out)[v] = make_float4(y[0], y[1], y[2], y[3]);
            } else {
              const __nv_bfloat162 ya = __floats2bfloat162_rn(y[0], y[1]), yb = __floats2bfloat162_rn(y[2], y[3]);
              reinterpret_cast<uint2*>(out)[v] =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&ya), *reinterpret_cast<const uint32_t*>(&yb));
            }
          }
          if (a.lse && r == 0 && pw == 0)
            a.lse[orow] = l == 0.f ? -INFINITY : (w.m[nt][x] + (log2f(l) - kBias)) * 0.69314718055994531f;
        } else {
          const long long at_row = slot * L.rows_pass + (row - pass0);
          float4* o = reinterpret_cast<float4*>(L.o + at_row * D + d0);
#pragma unroll
          for (int v = 0; v < kOwn / 4; ++v)
            o[v] = make_float4(w.o[2 * v][nt][x], w.o[2 * v][nt][2 + x], w.o[2 * v + 1][nt][x], w.o[2 * v + 1][nt][2 + x]);
          if (r == 0 && pw == 0) L.ml[at_row] = make_float2(w.m[nt][x], l);
        }
      }
    if (first == 0) {
      // rows past the request's own (all of them if its lengths are bad)
      if (sp.bad && at.hr == 0 && first_warp && lane == 0) atomicOr(a.status, 1 << SSD_ERR_LENGTH);
      const float none = sp.bad ? __int_as_float(0x7FC00000) : 0.f;
      const int end = min(pass0 + L.rows_pass, L.rows);
      for (int row = max(pass0, nrows) + group * P + pw; row < end; row += G * P) {
        const long long orow = (static_cast<long long>(b) * a.nq + row / L.per) * a.heads + h * L.per + row % L.per;
        for (int d = lane; d < D; d += 32) static_cast<E*>(a.out)[orow * D + d] = static_cast<E>(none);
        if (a.lse && lane == 0) a.lse[orow] = sp.bad ? none : -INFINITY;
      }
    }
    at.tile += count;
    if (at.tile == at.s.tiles) {
      at.tile = at.s.tiles - 1;
      at.next(a, list.per_request);
    }
  }
  if (dead) {
    // say so, and give the copies still in flight the same time again before
    // the shared memory goes
    if (lane == 0) atomicOr(a.status, 1 << SSD_ERR_CUDA);
    bar_wait(bars + (team * S + (take + S - 1) % S) * 16, take ? phase : phase ^ 1);
  }
}

template <typename E, int D, int NT, int P>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_kernel(const __grid_constant__ AttnLaunch L) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long scan[kThreads], sums[kThreads / 32];
  __shared__ int2 spans[kWarps][NT * 8];
  const KvAttnArgs& a = L.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bars = smem_u32(smem), data = bars + kHead;
  volatile int* flags = reinterpret_cast<int*>(smem + 16 * kMaxStages);  // the stage lacks a bad page's block
  if (tid < L.p.t * L.p.s) {
    bar_init(bars + tid * 16, 1);
    bar_init(bars + tid * 16 + 8, P * L.p.g);
    flags[tid] = 0;
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  List<kTile> list;
  list.build(a, a.c.kv_heads * L.p.rt, gridDim.x * L.p.t, kPartTiles, scan, sums);
  // 128 x (224 + 224 + 56) registers: the 384 x 168 of the launch
  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kWarps) produce<D>(L, list, bars, data, flags, lane);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    if (warp < L.p.t * L.p.g * P) consume<E, D, NT, P>(L, list, bars, data, flags, spans[warp], warp, lane);
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
  if (local >= L.rows_pass || row >= nrows) return;
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

template <typename E, int D>
cudaError_t launch_join(const AttnLaunch& L, int sms, cudaStream_t s) {
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

template <typename E, int D, int NT, int P>
cudaError_t launch_shape(const AttnLaunch& L, int sms, cudaStream_t s) {
  const int smem = kHead + L.p.t * (L.p.s * stage_bytes(D) + (P == 2 ? L.p.g * pair_bytes(D, NT, sizeof(E) == 4) : 0));
  cudaError_t e = allow_shared<kv_attention_kernel<E, D, NT, P>>(kSmem);
  if (e != cudaSuccess) return e;
  kv_attention_kernel<E, D, NT, P><<<sms, kThreads, smem, s>>>(L);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<E, D>(L, sms, s);
}

template <typename E, int D, int P, int NT>
cudaError_t launch_rows(const AttnLaunch& L, int sms, cudaStream_t s) {
  constexpr bool kF32 = sizeof(E) == 4;
  if constexpr (NT <= max_nt(D, kF32, P) && (P == 1 || NT >= (kF32 || D == 256 ? 1 : 3))) {
    if (L.p.nt == NT) return launch_shape<E, D, NT, P>(L, sms, s);
  }
  if constexpr (NT > 1) return launch_rows<E, D, P, NT - 1>(L, sms, s);
  return cudaErrorInvalidValue;
}

template <typename E, int D>
cudaError_t launch_dim(const AttnLaunch& L, int sms, cudaStream_t s) {
  if (L.p.p == 1) return launch_rows<E, D, 1, 2>(L, sms, s);
  if constexpr (D == 128 && sizeof(E) == 2) return cudaErrorInvalidValue;  // rows for pairs go to ssdv_attn_tc.cu
  else return launch_rows<E, D, 2, 6>(L, sms, s);
}

struct WorkLayout {
  size_t desc, ml, o, total;
};
WorkLayout work_layout(const AttnShape& p, int D) {
  WorkLayout w;
  const size_t teams = static_cast<size_t>(kMaxSms) * p.t, rows = 2 * teams * p.g * p.nt * 8;
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
  L.rows_pass = L.p.g * L.p.nt * 8;
  const WorkLayout w = work_layout(L.p, D);
  L.desc = reinterpret_cast<int4*>(a.work + w.desc);
  L.ml = reinterpret_cast<float2*>(a.work + w.ml);
  L.o = reinterpret_cast<float*>(a.work + w.o);
  if (L.p.tc) {
    e = launch_attention_tc(L, sms, stream);
    return e == cudaSuccess ? launch_join<__nv_bfloat16, 128>(L, sms, stream) : e;
  }
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
