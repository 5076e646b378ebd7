// ssdv_kv.cu -- writing keys and values into the 4-bit cache and reading them
// back (layout and numbers: ssdv_kv.cuh).
//
// One thread takes one group (16 elements of a head) of 8 tokens of one block,
// for keys or for values.  The lanes of a warp take neighbouring groups, so
// that each token's row is read and written in whole sectors.  A key row's words
// come from one token; the 8 tokens of a value word are the thread's own, and the
// two threads of a block's halves exchange words so that each writes 16 bytes at
// a time.  A block belongs to one request, so a value word that also holds tokens
// of earlier calls is updated by one thread.
//
// Both are bound by memory; what they compute per element is kept to a few
// operations: quotients by a two-term reciprocal, the integer in the low bits of a
// sum with 1.5 * 2^23, places in the word by one multiply-add each (append), and
// fp16 pairs as in the attention (read).  Measured, 8 prompts of 701 to 4099 bf16
// tokens, 8 heads of 128: writing 19.5 us for 24 MB of rows (a chain of loads, the
// lengths, the page table, the rows, and about 200 instructions a group at 0.5 a
// cycle), reading 22 us for 134 MB with the rows past a request's count (the copy
// bandwidth).  300 requests of up to 41 tokens, 2 heads of 256: 13 and 8.5 us (16.5
// for writing with its loops unrolled).
#include "ssdv_kv.cuh"

namespace ssdv {

namespace {

constexpr int kThreads = 128;

// A group as it lies in memory: 8 words of bf16 pairs, or 16 fp32 numbers.
template <typename E>
struct Raw {
  static constexpr int kWords = sizeof(E) * 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const E* p, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (sizeof(E) == 2) {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = h[2 * i] | static_cast<uint32_t>(h[2 * i + 1]) << 16;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(static_cast<float>(p[i]));
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(E) == 2) return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    else return __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void limit(float most) {  // NaN becomes `most` too
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(E) == 2) {  // most, 7 times a scale, fits bf16
        const uint32_t lo = __float_as_uint(fminf(fmaxf(at(2 * i), -most), most));
        const uint32_t hi = __float_as_uint(fminf(fmaxf(at(2 * i + 1), -most), most));
        w[i] = lo >> 16 | (hi & 0xFFFF0000u);
      } else {
        w[i] = __float_as_uint(fminf(fmaxf(at(i), -most), most));
      }
    }
  }
  // Bits of the largest magnitude; above 0x7F800000 if there is a NaN.
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = 0;
    if constexpr (sizeof(E) == 2) {
      uint32_t x = 0;  // both halves of the words at once
#pragma unroll
      for (int i = 0; i < 8; ++i) x = __vmaxu2(x, w[i] & 0x7FFF7FFFu);
      m = max(x << 16, x & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    }
    return m;
  }
};

constexpr float kMagic = 12582920.f;          // 1.5 * 2^23 + 8: the sum's low bits are n + 8
constexpr uint32_t kMagicBits = 0x4B400000u;  // without the 8

// A group's scale byte, and its codes n + 8 as kMagicBits + (n + 8).  x / s comes
// from 1/s in two terms (r + e, good to 2^-46): a quotient that is a tie between two
// integers comes out exactly, and any other lies more than half an ulp away from
// one.  |x| / s stays below 7.5 (a scale is rounded down by one part in 17 at
// most), but for scales of fewer bits (byte < 8) and beyond the largest.
template <typename E>
__device__ __forceinline__ uint32_t quantise(Raw<E>& x, uint32_t (&u)[16]) {
  const uint32_t top = x.largest();
  const bool nan = top > 0x7F800000u;
  const uint32_t byte = nan ? 0u : kv_scale_byte(__uint_as_float(top));
  const float s = kv_scale(byte);
  if (byte < 8 || byte == kKvMaxScaleByte) x.limit(7.f * s);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(byte ? s : 1.f));
  const float e = fmaf(-s, r, 1.0f) * r;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = x.at(i);
    u[i] = __float_as_uint(fmaf(v, r, v * e) + kMagic);
  }
  return nan ? kKvNanByte : byte;
}

// Where entry e of a word lies, counting from the rotation that entries 4 to 7 get,
// and what kMagicBits adds up to over four entries.
__host__ __device__ constexpr uint32_t entry_unit(int e) { return 1u << (((e >> 1) & 1 ? 2 : 6) + ((e & 1) << 4)); }
constexpr uint32_t kMagicFour = kMagicBits * (entry_unit(0) + entry_unit(1) + entry_unit(2) + entry_unit(3));
__device__ __forceinline__ uint32_t turn(uint32_t w) { return __funnelshift_l(w, w, 8); }

// The thread's task: its request, block, head, token half and group, and the
// tokens [t0, t1) of the block that the call covers.
struct Task {
  int b, h, half, g, t0, t1;
  long long first;  // index of the block's token 0 among the call's tokens (may be negative)
  uint8_t* block;   // null: nothing to do here
  bool bad;
};

template <int D>
__device__ __forceinline__ Task find_task(const KvStoreArgs& a) {
  constexpr int G = D / 16;
  Task k;
  k.block = nullptr;
  k.bad = false;
  const int nblk = (a.n + 2 * kKvBlock - 2) / kKvBlock;  // blocks that n tokens may touch
  long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  k.g = static_cast<int>(id % G);
  id /= G;
  k.half = static_cast<int>(id & 1);
  id >>= 1;
  k.h = static_cast<int>(id % a.c.kv_heads);
  id /= a.c.kv_heads;
  const int j = static_cast<int>(id % nblk);
  id /= nblk;
  k.t0 = k.t1 = 0;
  k.first = 0;
  if (id >= a.B) {
    k.b = -1;
    return k;
  }
  k.b = static_cast<int>(id);
  const int start = a.start[k.b];
  const int count = a.count ? a.count[k.b] : a.n;
  const bool lead = j == 0 && k.h == 0 && k.half == 0 && k.g == 0 && blockIdx.y == 0;
  if (start < 0 || count < 0 || count > a.n ||
      static_cast<long long>(start) + count > static_cast<long long>(a.c.max_pages) * a.c.page_size) {
    if (lead) atomicOr(a.status, 1 << SSD_ERR_LENGTH);
    k.bad = true;
    k.first = static_cast<long long>(j) * kKvBlock;  // the read kernel marks all n rows
    k.t0 = 0;
    k.t1 = kKvBlock;
    return k;
  }
  const long long pos0 = (static_cast<long long>(start) / kKvBlock + j) * kKvBlock;
  k.first = pos0 - start;
  k.t0 = k.first < 0 ? static_cast<int>(-k.first) : 0;
  const long long left = count - k.first;
  k.t1 = left < kKvBlock ? (left > 0 ? static_cast<int>(left) : 0) : kKvBlock;
  if (k.t0 >= k.t1) return k;
  const int page = a.c.page_table[static_cast<long long>(k.b) * a.c.max_pages + pos0 / a.c.page_size];
  if (page < 0 || page >= a.c.n_pages) {
    if (k.h == 0 && k.half == 0 && k.g == 0 && blockIdx.y == 0) atomicOr(a.status, 1 << SSD_ERR_PAGE);
    k.bad = true;
    return k;
  }
  const int per = a.c.page_size / kKvBlock;
  const long long at = (static_cast<long long>(page) * a.c.kv_heads + k.h) * per + (pos0 / kKvBlock) % per;
  k.block = a.c.pages + at * kv_block_bytes(D);
  return k;
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvStoreArgs a, int vec) {
  constexpr int G = D / 16, kBatch = sizeof(E) == 2 ? 2 : 1;  // tokens at a time, as many on their way
  const Task k = find_task<D>(a);
  const int lo = max(k.t0, k.half * 8), hi = k.block ? min(k.t1, k.half * 8 + 8) : 0;
  const bool values = blockIdx.y != 0;
  const long long* st = values ? a.vs : a.ks;
  const E* base = static_cast<const E*>(values ? a.v : a.k) + k.b * st[0] + k.h * st[2] + k.g * 16;
  Raw<E> next[kBatch];
  const auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = k.half * 8 + i0 + i;
      if (t >= lo && t < hi) next[i].load(base + (k.first + t) * st[1], vec);
    }
  };
  // (loops stay rolled: a small call runs code that is in no cache yet)
  if (!values) {
    load(0);
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += kBatch) {
      Raw<E> x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) x[i] = next[i];
      if (i0 + kBatch < 8) load(i0 + kBatch);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = k.half * 8 + i0 + i;
        if (t < lo || t >= hi) continue;
        uint32_t u[16], word[2];
        const uint32_t byte = quantise(x[i], u);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t w = 0u - kMagicFour;
#pragma unroll
          for (int e = 4; e < 8; ++e) w += u[8 * j + e] * entry_unit(e);
          w = turn(w) - kMagicFour;
#pragma unroll
          for (int e = 0; e < 4; ++e) w += u[8 * j + e] * entry_unit(e);
          word[j] = w;
        }
        *reinterpret_cast<uint2*>(k.block + k_word_offset<D>(t, 2 * k.g)) = make_uint2(word[0], word[1]);
        k.block[k_scale_offset<D>(t, k.g)] = static_cast<uint8_t>(byte);
      }
    }
    return;
  }
  uint32_t word[16] = {}, keep = 0xFFFFFFFFu;
  load(4);
#pragma unroll 1
  for (int n = 0; n < 8; n += kBatch) {
    const int i0 = (n + 4) & 7;  // tokens 4 to 7 first: theirs are turned
    Raw<E> x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) x[i] = next[i];
    if (n + kBatch < 8) load((i0 + kBatch) & 7);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = k.half * 8 + i0 + i;
      if (t < lo || t >= hi) continue;
      uint32_t u[16];
      const uint32_t byte = quantise(x[i], u), unit = entry_unit(i0 + i);
#pragma unroll
      for (int d = 0; d < 16; ++d) word[d] += (u[d] - kMagicBits) * unit;
      keep &= ~kv_place(15u, i0 + i);
      k.block[kv_v_scales(D) + k.g * kKvBlock + t] = static_cast<uint8_t>(byte);
    }
    if (n + kBatch == 4) {
#pragma unroll
      for (int d = 0; d < 16; ++d) word[d] = turn(word[d]);
    }
  }
  // the halves' threads exchange: each gets 8 elements' words of both halves
  const uint32_t other_keep = __shfl_xor_sync(~0u, keep, G);
  uint32_t get[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) get[d] = __shfl_xor_sync(~0u, k.half ? word[d] : word[8 + d], G);
  const uint32_t keep0 = k.half ? other_keep : keep, keep1 = k.half ? keep : other_keep;
  if (!k.block || (keep0 == 0xFFFFFFFFu && keep1 == 0xFFFFFFFFu)) return;
#pragma unroll
  for (int d = 0; d < 8; d += 2) {  // elements 8 half + d and the next: 16 bytes
    uint4* p = reinterpret_cast<uint4*>(k.block + v_word_offset<D>(k.g * 16 + k.half * 8 + d, 0));
    uint4 v = k.half ? make_uint4(get[d], word[8 + d], get[d + 1], word[9 + d])
                     : make_uint4(word[d], get[d], word[d + 1], get[d + 1]);
    if (keep0 | keep1) {
      const uint4 old = *p;
      v.x |= old.x & keep0, v.y |= old.y & keep1, v.z |= old.z & keep0, v.w |= old.w & keep1;
    }
    *p = v;
  }
}

// Two codes of a word (pair p of four) times their scales, as fp32.
__device__ __forceinline__ float2 pair_values(uint32_t word, int p, uint32_t scale) {
  const uint32_t w = p & 2 ? __funnelshift_r(word, word, 8) : word;
  const uint32_t x = p & 1 ? (w & 0x003C003Cu) | 0x5C005C00u : (w & 0x03C003C0u) | 0x4C004C00u;
  uint32_t by, y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(by) : "r"(scale), "r"(p & 1 ? 0xDC20DC20u : 0xCE00CE00u));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(scale), "r"(by));
  return __half22float2(*reinterpret_cast<const __half2*>(&y));
}

// wide: p is 32-byte aligned.  One store then covers whole sectors; two of 16 bytes
// each touch every sector twice (8 prompts of 701 to 4099 tokens: 22 against 35 us).
__device__ __forceinline__ void store32(void* p, uint4 a, uint4 b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = a;
    static_cast<uint4*>(p)[1] = b;
  }
}

template <typename E>
__device__ __forceinline__ void store_group(E* p, const float (&x)[16], bool wide) {
  if constexpr (sizeof(E) == 2) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    store32(p, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]), wide);
  } else {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                        __float_as_uint(x[4 * i + 3]));
    store32(p, w[0], w[1], wide);
    store32(p + 8, w[2], w[3], wide);
  }
}

// Rows past a request's count are zero; rows of a request in error are NaN.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvStoreArgs a, bool wide) {
  const Task k = find_task<D>(a);
  if (k.b < 0) return;
  const bool values = blockIdx.y != 0;
  const long long row = static_cast<long long>(a.c.kv_heads) * D;
  E* out = static_cast<E*>(values ? a.out_v : a.out_k) +
           (static_cast<long long>(k.b) * a.n * a.c.kv_heads + k.h) * D + k.g * 16 + k.first * row;
  const int first = static_cast<int>(max(-k.first, 0ll));  // tokens of the block that have a row
  const int last = static_cast<int>(min(static_cast<long long>(a.n) - k.first, static_cast<long long>(kKvBlock)));
  if (!k.block) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = k.half * 8 + i;
      const bool live = t >= k.t0 && t < k.t1;
#pragma unroll
      for (int d = 0; d < 16; ++d) x[d] = k.bad && live ? __int_as_float(0x7FC00000) : 0.f;
      if (t >= first && t < last) store_group(out + t * row, x, wide);
    }
    return;
  }
  if (!values) {
    uint2 w[8];
    uint32_t sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = k.half * 8 + i;
      w[i] = *reinterpret_cast<const uint2*>(k.block + k_word_offset<D>(t, 2 * k.g));
      sc[i] = k.block[k_scale_offset<D>(t, k.g)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = k.half * 8 + i;
      float x[16];
      const bool live = t >= k.t0 && t < k.t1;
      const uint32_t scale = sc[i] * 0x00800080u;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float2 f = pair_values(p < 4 ? w[i].x : w[i].y, p & 3, scale);
        x[2 * p] = live ? f.x : 0.f, x[2 * p + 1] = live ? f.y : 0.f;
      }
      if (t >= first && t < last) store_group(out + t * row, x, wide);
    }
    return;
  }
  uint32_t vw[16];
#pragma unroll
  for (int d = 0; d < 16; ++d) vw[d] = *reinterpret_cast<const uint32_t*>(k.block + v_word_offset<D>(k.g * 16 + d, k.half));
  const uint2 sv = *reinterpret_cast<const uint2*>(k.block + kv_v_scales(D) + k.g * kKvBlock + k.half * 8);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int t = k.half * 8 + 2 * p;
    const uint32_t scale = __byte_perm(p < 2 ? sv.x : sv.y, 0, p & 1 ? 0x4342 : 0x4140) << 7;
    const bool live0 = t >= k.t0 && t < k.t1, live1 = t + 1 >= k.t0 && t + 1 < k.t1;
    float x[16], y[16];
#pragma unroll
    for (int d = 0; d < 16; ++d) {
      const float2 f = pair_values(vw[d], p, scale);
      x[d] = live0 ? f.x : 0.f, y[d] = live1 ? f.y : 0.f;
    }
    if (t >= first && t < last) store_group(out + t * row, x, wide);
    if (t + 1 >= first && t + 1 < last) store_group(out + (t + 1) * row, y, wide);
  }
}

long long tasks(const KvStoreArgs& a, int D) {
  const long long nblk = (a.n + 2 * kKvBlock - 2) / kKvBlock;
  return a.B * nblk * a.c.kv_heads * 2 * (D / 16);
}

template <typename E>
cudaError_t append_dim(const KvStoreArgs& a, int D, int vec, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((tasks(a, D) + kThreads - 1) / kThreads), 2);
  if (D == 64) kv_append_kernel<E, 64><<<grid, kThreads, 0, s>>>(a, vec);
  else if (D == 128) kv_append_kernel<E, 128><<<grid, kThreads, 0, s>>>(a, vec);
  else kv_append_kernel<E, 256><<<grid, kThreads, 0, s>>>(a, vec);
  return cudaGetLastError();
}

template <typename E>
cudaError_t read_dim(const KvStoreArgs& a, int D, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((tasks(a, D) + kThreads - 1) / kThreads), 2);
  const bool wide = (reinterpret_cast<uintptr_t>(a.out_k) | reinterpret_cast<uintptr_t>(a.out_v)) % 32 == 0;
  if (D == 64) kv_read_kernel<E, 64><<<grid, kThreads, 0, s>>>(a, wide);
  else if (D == 128) kv_read_kernel<E, 128><<<grid, kThreads, 0, s>>>(a, wide);
  else kv_read_kernel<E, 256><<<grid, kThreads, 0, s>>>(a, wide);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvStoreArgs& a, int D, int esize, bool vec, cudaStream_t stream) {
  return esize == 2 ? append_dim<__nv_bfloat16>(a, D, vec, stream) : append_dim<float>(a, D, vec, stream);
}

cudaError_t launch_kv_read(const KvStoreArgs& a, int D, int esize, cudaStream_t stream) {
  return esize == 2 ? read_dim<__nv_bfloat16>(a, D, stream) : read_dim<float>(a, D, stream);
}

}  // namespace ssdv
