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
// A CTA takes a token: its threads share out the sines and cosines, then its warps the
// heads.  D / 16 lanes take a head's row, 16 elements a lane as two vectors that hold
// eight pairs whole, so a pair never crosses lanes; up to four rows a lane are loaded
// before the first is used.
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

// (x, y) *= (a, b); (x, y) += (a, b)^2: two fp32 operations at once.
__device__ __forceinline__ void mul_pair(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void add_squares(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "fma.rn.f32x2 a, b, b, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// The rows of queries or of keys of a token.
template <typename E, int D, bool kInterleaved, bool kVec>
__device__ __forceinline__ void turn_rows(const E* in, E* out, long long stride, long long out_stride, int heads,
                                          const float* weight, float eps, bool real, float fill, bool turned, int d0, int d1,
                                          const float* cosines, int warp, int lane) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes, kStep = kThreads / 32 * kGroups;
  const int first = warp * kGroups + lane / kLanes;
  float w[16];
#pragma unroll 1
  for (int j0 = 0; j0 < heads; j0 += kStep * kRows) {
    float x[kRows][16];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int j = j0 + r * kStep + first;
      if (real && j < heads) {
        load8<E, kVec>(in + j * stride + d0, x[r]);
        load8<E, kVec>(in + j * stride + d1, x[r] + 8);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[r][e] = fill;
      }
    }
    if (j0 == 0) {
      __syncthreads();  // (the sines are there)
      if (weight) {
        load8<float, true>(weight + d0, w);
        load8<float, true>(weight + d1, w + 8);
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (j0 + r * kStep >= heads) break;  // (the CTA agrees)
      const int j = j0 + r * kStep + first;
      if (weight && real) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int e = 0; e < 16; e += 2) add_squares(a, b, x[r][e], x[r][e + 1]);
        a += b;
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) a += __shfl_xor_sync(~0u, a, o);
        const float inv = 1.f / sqrtf(a * (1.f / D) + eps);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          mul_pair(x[r][e], x[r][e + 1], inv, inv);
          mul_pair(x[r][e], x[r][e + 1], w[e], w[e + 1]);
        }
      }
      if (turned && real) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& p = x[r][kInterleaved ? 2 * e : e];
          float& q = x[r][kInterleaved ? 2 * e + 1 : e + 8];
          const float2 t = reinterpret_cast<const float2*>(cosines)[e];
          const float y = p * t.x - q * t.y;
          q = p * t.y + q * t.x;
          p = y;
        }
      }
      if (j < heads) {
        store8<E, kVec>(out + j * out_stride + d0, x[r]);
        store8<E, kVec>(out + j * out_stride + d1, x[r] + 8);
      }
    }
  }
}

template <typename E, int D, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float2 turn[D / 2];  // cosine and sine of each pair
  const int tid = threadIdx.x, lane = tid & 31, l = lane % (D / 16), warp = tid >> 5;
  const int b = blockIdx.x / a.n, i = blockIdx.x - b * a.n;
  const int len = a.len[b], count = a.n_new ? a.n_new[b] : a.n;
  const bool bad = len < 0 || count < 0 || count > a.n || static_cast<long long>(len) + count > (1ll << 30);
  if (bad && i == 0 && tid == 0) atomicOr(a.status, 1 << SSD_ERR_LENGTH);
  const bool real = !bad && i < count;
  if (real && tid < a.rot / 2) {
    const float freq = a.freq[tid];
    const unsigned long long t = turns(freq) * static_cast<unsigned long long>(static_cast<unsigned>(len + i));
    float2 y;
    sincospif(__ll2float_rn(static_cast<long long>(t)) * 1.0842021724855044e-19f, &y.y, &y.x);  // 2^-63
    if (!isfinite(freq)) y.x = y.y = __int_as_float(0x7FC00000);
    turn[tid] = y;
  }
  // the lane's two vectors: of the rotated pairs' first and second halves, or side by side
  const bool turned = l < a.rot / 16, apart = !kInterleaved && turned;
  const int d0 = apart ? 8 * l : 16 * l, d1 = apart ? 8 * l + a.rot / 2 : 16 * l + 8;
  const float fill = bad ? __int_as_float(0x7FC00000) : 0.f;
  const float* mine = reinterpret_cast<const float*>(turn + (turned ? 8 * l : 0));
  turn_rows<E, D, kInterleaved, kVec>(static_cast<const E*>(a.q) + b * a.qs[0] + i * a.qs[1],
                                      static_cast<E*>(a.out_q) + b * a.oqs[0] + i * a.oqs[1], a.qs[2], a.oqs[2], a.heads,
                                      a.q_weight, a.eps, real, fill, turned, d0, d1, mine, warp, lane);
  if (a.kv_heads)
    turn_rows<E, D, kInterleaved, kVec>(static_cast<const E*>(a.k) + b * a.ks[0] + i * a.ks[1],
                                        static_cast<E*>(a.out_k) + b * a.oks[0] + i * a.oks[1], a.ks[2], a.oks[2],
                                        a.kv_heads, a.k_weight, a.eps, real, fill, turned, d0, d1, mine, warp, lane);
}

template <typename E, int D>
cudaError_t launch_dim(const RopeArgs& a, bool interleaved, bool vec, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(a.B) * a.n);
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
