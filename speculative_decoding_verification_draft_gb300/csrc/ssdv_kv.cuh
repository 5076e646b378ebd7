// ssdv_kv.cuh -- the 4-bit key/value cache: its layout, its numbers and the
// launch arguments of its kernels (ssdv_kv.cu: append and read; ssdv_attn.cu:
// attention).
//
// Numbers.  16 consecutive elements of a head's row form a group with scale
//   s = RN_E5M3(max|x| / 7)   (at most 240)
// and integers n = clamp(RN(x / s), -7, 7), both to the nearest, ties to even.
// E5M3 is the upper byte of an fp16 number whose sign is dropped: fp16 bits =
// byte << 7, so 4 bits of significand, multiples of 2^-17 below 2^-14.  n s
// has 7 bits of significand: exact in bf16 and fp16.  0xFF marks a group that
// held a NaN (fp16 NaN); an infinity saturates (s = 240, n = +-7).
// The fp32 quotients round as the real ones: every border (k + 1/2) s, and 7
// times a border of E5M3, has few bits, so the fp32 numbers next to it lie
// more than half an ulp of the quotient away from it.
//
// Layout.  Page p holds for each kv head page_size / 16 blocks of 16 tokens,
// 18 D bytes each, ordered for the attention kernel's matrix fragments:
//   K codes  [16 tokens][D / 2 bytes]: word w of a row holds elements 8 w ..;
//            at D = 256 the two 64-byte halves of odd tokens are exchanged
//            (shared-memory banks)
//   V codes  [D / 16][8][2][16 tokens x 4 bits]: entry (i, r, e) is element
//            r D/8 + 2 i + e; word 0 tokens 0..7, word 1 tokens 8..15
//   K scales, D bytes: for each 8 groups 4 pairs of groups, for each pair the
//            even tokens' two scales, then the odd tokens' (D = 64: 4 groups, for
//            each the even tokens' scale, then the odd tokens')
//   V scales [D / 16][16 tokens]
// A word holds 8 codes n + 8 as four pairs, pair p = entries 2p (low half-word)
// and 2p + 1 (high): pair 0 at bits 9:6 of each half-word and pair 1 at bits
// 5:2; pairs 2 and 3 the same after a rotation right by 8.  Or-ing 0x4C00 to
// bits 9:6 gives the fp16 number 16 + (n + 8), or-ing 0x5C00 to bits 5:2 gives
// 256 + (n + 8): one logic operation and one fused multiply-add per pair
// ((16 + n + 8) s - 24 s, (256 + n + 8) s - 264 s, every term exact for
// s <= 240) give two values n s.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssdv.h"

namespace ssdv {

constexpr int kKvBlock = 16;           // tokens per block, elements per group
constexpr int kKvMaxScaleByte = 183;   // 240
constexpr int kKvNanByte = 0xFF;

__host__ __device__ constexpr int kv_block_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int kv_v_codes(int D) { return 8 * D; }
__host__ __device__ constexpr int kv_k_scales(int D) { return 16 * D; }
__host__ __device__ constexpr int kv_v_scales(int D) { return 17 * D; }

struct KvCacheArgs {
  uint8_t* pages;
  long long n_pages;
  int kv_heads, page_size, max_pages;
  const int32_t* page_table;  // [B, max_pages]
};

struct KvStoreArgs {
  KvCacheArgs c;
  const int32_t* start;  // [B]: position of the request's first token
  const int32_t* count;  // [B] or null (n tokens each)
  int B, n;
  const void* k;
  const void* v;
  long long ks[3], vs[3];  // append: element strides of request, token, head
  void* out_k;             // read: [B, n, kv_heads, D]
  void* out_v;
  int32_t* status;
};
cudaError_t launch_kv_append(const KvStoreArgs& a, int D, int esize, bool vec, cudaStream_t stream);
cudaError_t launch_kv_read(const KvStoreArgs& a, int D, int esize, cudaStream_t stream);

struct KvAttnArgs {
  KvCacheArgs c;
  const int32_t* kv_len;  // [B]
  const int32_t* n_q;     // [B] or null (nq each)
  int B, nq, heads;
  const void* q;
  long long qs[3];        // element strides of request, token, head
  float scale_log2;       // scale * log2(e)
  int window;             // 0: none
  int sinks;              // with a window: the first positions stay visible (0: none)
  int past_only;
  const int32_t* first;   // [B] or null: positions below first[b] are left out (without sinks)
  void* out;              // [B, nq, heads, D]
  float* lse;             // [B, nq, heads] or null
  float2* own_ml;         // in place of out and lse, or null: [B, kv_heads, nq * heads / kv_heads] maximum and sum
  float* own_o;           // and [.., D] sums of the rows that are real, as parts keep them;
  int2* own_parts;        // [B, kv_heads, passes]: parts of the pass's rows and the first's slot.  Rows in
                          // more parts than one are not in own_ml and own_o but where own_slots says
  int32_t* status;
  uint8_t* work;          // partial results
};
cudaError_t launch_kv_attention(const KvAttnArgs& a, int D, int esize, cudaStream_t stream);
size_t kv_attention_work_bytes(int rows, int D);
// Where a call with own_parts leaves the parts of rows in several: part k of row r of a
// pass is at (k ? 2 (slot / 2 + k) : slot) * rows_pass + r.
struct OwnSlots {
  const float2* ml;
  const float* o;
  int rows_pass, passes;
};
OwnSlots kv_own_slots(const KvAttnArgs& a, int D, int esize);
// The same for groups of requests that share a prefix (ssdv_shared.cu).
cudaError_t launch_kv_shared(const KvAttnArgs& a, const int32_t* group_start, const int32_t* shared_len, int G, int D,
                             int esize, cudaStream_t stream);
size_t kv_shared_work_bytes(int B, int nq, int heads, int kv_heads, int D, int G);

#ifdef __CUDACC__

// Byte offset of K word w of token t in a block.
template <int D>
__device__ __forceinline__ int k_word_offset(int t, int w) {
  const int x = D == 256 ? ((t & 1) << 4) : 0;
  return t * (D / 2) + ((w ^ x) << 2);
}
// Byte offset of the V word of element d, tokens 8 half .. 8 half + 7.
template <int D>
__device__ __forceinline__ int v_word_offset(int d, int half) {
  constexpr int per = D / 8;
  const int r = d / per, i = (d % per) >> 1, e = d & 1;
  return kv_v_codes(D) + (((i * 8 + r) * 2 + e) << 3) + (half << 2);
}

// Byte offset of the K scale of token t, group g.
template <int D>
__device__ __forceinline__ int k_scale_offset(int t, int g) {
  const int at = D == 64 ? g * 16 + (t & 1) * 8 + (t >> 1) : (g >> 1) * 32 + (t & 1) * 16 + (t >> 1) * 2 + (g & 1);
  return kv_k_scales(D) + at;
}

// Code u (0..15) of entry e in its word, and back.
__device__ __forceinline__ uint32_t kv_place(uint32_t u, int e) {
  const int p = e >> 1;
  uint32_t x = u << (((p & 1) ? 2 : 6) + ((e & 1) << 4));
  return p & 2 ? __funnelshift_l(x, x, 8) : x;
}
__device__ __forceinline__ int kv_code(uint32_t w, int e) {
  const int p = e >> 1;
  const uint32_t x = p & 2 ? __funnelshift_r(w, w, 8) : w;
  return static_cast<int>((x >> (((p & 1) ? 2 : 6) + ((e & 1) << 4))) & 15u) - 8;
}
__device__ __forceinline__ float kv_scale(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// max|x| / 7 to the scale byte (x without NaN).  The quotient is taken with 1/7 in
// two terms, good to 2^-47: a tie of the scale's 4 bits comes out exactly.
__device__ __forceinline__ uint32_t kv_scale_byte(float amax) {
  constexpr float kSeventh = 1.0f / 7.0f, kRest = static_cast<float>(1.0 / 7.0 - kSeventh);
  const float x = fminf(amax, 1680.0f), f = fmaf(x, kSeventh, x * kRest);
  if (f < 6.103515625e-05f)  // below 2^-14: multiples of 2^-17 (64 has that ulp)
    return __float_as_uint(f + 64.0f) - __float_as_uint(64.0f);
  const uint32_t u = __float_as_uint(f);
  const uint32_t r = u + 0x7FFFFu + ((u >> 20) & 1u);  // to 3 bits of fraction, ties to even
  const uint32_t b = (r >> 20) - ((127u - 15u) << 3);
  return b < kKvMaxScaleByte ? b : kKvMaxScaleByte;
}

#endif  // __CUDACC__

}  // namespace ssdv
