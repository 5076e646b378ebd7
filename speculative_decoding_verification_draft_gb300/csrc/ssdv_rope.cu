// ssdv_rope.cu -- norms of queries and keys for each head, and the rotation by
// position, in one pass.
//
//   y = x * w / sqrt(mean x^2 + eps)
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_a sin t + y_b cos t),  t = position * freq_i
// for the rot / 2 pairs (a, b) = (i, i + rot / 2), or (2i, 2i + 1) interleaved.
//
// Angles are exact whatever the position: freq / 2 pi is held as a 64-bit fraction
// of a turn (to 2^-64), position times that wraps around by itself, and what is
// left goes to fp32 in half-turns.  An angle is off by 2^-24 of itself and by
// position * 2^-63 half-turns.
//
// D / 16 lanes take a head's row, 16 elements a lane as two vectors that hold the
// lane's eight pairs whole, so a pair never crosses lanes.  A warp takes one token
// and up to four rows of each of its groups of lanes, all loaded before the first
// is used; its lanes share out the token's sines and cosines.
#include <cuda_bf16.h>

#include "ssdv.h"
#include "ssdv_round.cuh"

namespace ssdv {

namespace {

constexpr int kThreads = 128, kRows = 4;

// A lane's 16 elements of a row: eight from d0, eight from d1.
template <typename E, bool kVec>
__device__ __forceinline__ void load8(const E* p, float* x) {
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(p[i]);
  } else if constexpr (sizeof(E) == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}
template <typename E, bool kVec>
__device__ __forceinline__ void store8(E* p, const float* x) {
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = static_cast<E>(x[i]);
  } else if constexpr (sizeof(E) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// freq / 2 pi modulo one turn, in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turns(float freq) {
  constexpr unsigned long long kInv = 0xA2F9836E4E44152Aull;  // 1 / 2 pi = kInv 2^-66
  const uint32_t u = __float_as_uint(freq);
  const int ex = (u >> 23) & 255;
  const unsigned long long m = ex ? (u & 0x7FFFFFu) | 0x800000u : u & 0x7FFFFFu;
  // m 2^(max(ex, 1) - 150) / 2 pi, in units of 2^-64
  const int shift = 152 - max(ex, 1);  // right, of m * kInv
  const unsigned long long hi = __umul64hi(m, kInv), lo = m * kInv;
  unsigned long long f = 0;
  if (shift >= 64) f = shift < 128 ? hi >> (shift - 64) : 0;
  else if (shift > 0) f = hi << (64 - shift) | lo >> shift;
  else if (shift > -64) f = lo << -shift;
  return u >> 31 ? 0ull - f : f;
}

template <typename E, int D, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes, kEach = 8 / kGroups;
  const int lane = threadIdx.x & 31, l = lane % kLanes, group = lane / kLanes;
  const int total = a.heads + a.kv_heads, per_token = (total + kGroups * kRows - 1) / (kGroups * kRows);
  const long long id = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const long long token = id / per_token;
  const int part = static_cast<int>(id - token * per_token);
  if (token >= static_cast<long long>(a.B) * a.n) return;
  const int b = static_cast<int>(token / a.n), i = static_cast<int>(token - static_cast<long long>(b) * a.n);
  const int len = a.len[b], count = a.n_new ? a.n_new[b] : a.n;
  const bool bad = len < 0 || count < 0 || count > a.n || static_cast<long long>(len) + count > (1ll << 30);
  if (bad && i == 0 && part == 0 && lane == 0) atomicOr(a.status, 1 << SSD_ERR_LENGTH);
  const bool real = !bad && i < count;
  // the lane's two vectors: of the rotated pairs' first and second halves, or side by side
  const bool turned = l < a.rot / 16;
  const bool apart = !kInterleaved && turned;
  const int d0 = apart ? 8 * l : 16 * l, d1 = apart ? 8 * l + a.rot / 2 : 16 * l + 8;

  const auto row = [&](int j, bool out) -> long long {
    const bool key = j >= a.heads;
    const long long* s = out ? (key ? a.oks : a.oqs) : (key ? a.ks : a.qs);
    return b * s[0] + i * s[1] + (key ? j - a.heads : j) * s[2];
  };
  float x[kRows][16];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int j = (part * kRows + r) * kGroups + group;
    if (real && j < total) {
      const E* p = static_cast<const E*>(j < a.heads ? a.q : a.k) + row(j, false);
      load8<E, kVec>(p + d0, x[r]);
      load8<E, kVec>(p + d1, x[r] + 8);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[r][e] = bad ? __int_as_float(0x7FC00000) : 0.f;
    }
  }
  // pair 8 l + e of the token: group g of lanes computes kEach of the lane's eight
  float c[8], s[8];
  {
    float mc[kEach], ms[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      mc[e] = 1.f, ms[e] = 0.f;
      if (turned && real) {
        const float freq = a.freq[8 * l + group * kEach + e];
        const unsigned long long t = turns(freq) * static_cast<unsigned long long>(static_cast<unsigned>(len + i));
        sincospif(__ll2float_rn(static_cast<long long>(t)) * 1.0842021724855044e-19f, &ms[e], &mc[e]);  // 2^-63
        if (!isfinite(freq)) mc[e] = ms[e] = __int_as_float(0x7FC00000);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = __shfl_sync(~0u, mc[e % kEach], e / kEach * kLanes + l);
      s[e] = __shfl_sync(~0u, ms[e % kEach], e / kEach * kLanes + l);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int j = (part * kRows + r) * kGroups + group;
    const float* w = j < a.heads ? a.q_weight : a.k_weight;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) sum = fmaf(x[r][e], x[r][e], sum);
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (j >= total) continue;
    if (w && real) {
      const float inv = 1.f / sqrtf(sum * (1.f / D) + a.eps);
      float v[16];
      load8<float, true>(w + d0, v);
      load8<float, true>(w + d1, v + 8);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[r][e] = x[r][e] * inv * v[e];
    }
    if (turned && real) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float& p = x[r][kInterleaved ? 2 * e : e];
        float& q = x[r][kInterleaved ? 2 * e + 1 : e + 8];
        const float y = p * c[e] - q * s[e];
        q = p * s[e] + q * c[e];
        p = y;
      }
    }
    E* out = static_cast<E*>(j < a.heads ? a.out_q : a.out_k) + row(j, true);
    store8<E, kVec>(out + d0, x[r]);
    store8<E, kVec>(out + d1, x[r] + 8);
  }
}

template <typename E, int D>
cudaError_t launch_dim(const RopeArgs& a, bool interleaved, bool vec, cudaStream_t stream) {
  constexpr int kGroups = 512 / D;
  const long long per_token = (a.heads + a.kv_heads + kGroups * kRows - 1) / (kGroups * kRows);
  const long long warps = per_token * a.B * a.n;
  const unsigned grid = static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32));
  if (interleaved) {
    if (vec) rope_kernel<E, D, true, true><<<grid, kThreads, 0, stream>>>(a);
    else rope_kernel<E, D, true, false><<<grid, kThreads, 0, stream>>>(a);
  } else {
    if (vec) rope_kernel<E, D, false, true><<<grid, kThreads, 0, stream>>>(a);
    else rope_kernel<E, D, false, false><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int D, int esize, bool interleaved, bool vec, cudaStream_t stream) {
  if (esize == 2) {
    if (D == 64) return launch_dim<__nv_bfloat16, 64>(a, interleaved, vec, stream);
    if (D == 128) return launch_dim<__nv_bfloat16, 128>(a, interleaved, vec, stream);
    return launch_dim<__nv_bfloat16, 256>(a, interleaved, vec, stream);
  }
  if (D == 64) return launch_dim<float, 64>(a, interleaved, vec, stream);
  if (D == 128) return launch_dim<float, 128>(a, interleaved, vec, stream);
  return launch_dim<float, 256>(a, interleaved, vec, stream);
}

}  // namespace ssdv
