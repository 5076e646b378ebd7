// ssdv_kv.cu -- writing keys and values into the 4-bit cache and reading them
// back (layout and numbers: ssdv_kv.cuh).
//
// One thread takes one group (16 elements of a head) of 8 tokens of one block,
// for keys or for values.  The lanes of a warp take neighbouring groups, so
// that each token's row is read and written in whole sectors, and no value
// crosses lanes: a key row's words come from one token, and the 8 tokens of a
// value word are the thread's own.  A block belongs to one request, so a value
// word that also holds tokens of earlier calls is updated by one thread.
#include "ssdv_kv.cuh"

namespace ssdv {

namespace {

constexpr int kThreads = 128;

template <typename E>
__device__ __forceinline__ void load_group(const E* p, bool vec, float (&x)[16]) {
  if (vec) {
    if constexpr (sizeof(E) == 2) {
      uint4 r[2];
      r[0] = __ldg(reinterpret_cast<const uint4*>(p));
      r[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
        x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = static_cast<float>(p[i]);
  }
}

// A group's scale byte and its codes n + 8 (0..15).
__device__ __forceinline__ uint32_t quantise(const float (&x)[16], uint32_t (&u)[16]) {
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    amax = fmaxf(amax, fabsf(x[i]));
    nan |= x[i] != x[i];
  }
  uint32_t byte = kv_scale_byte(amax);
  const float s = kv_scale(byte);
  const bool zero = byte == 0 || nan;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float n = fminf(fmaxf(rintf(x[i] / s), -7.f), 7.f);
    u[i] = zero ? 8u : static_cast<uint32_t>(static_cast<int>(n) + 8);
  }
  return nan ? kKvNanByte : byte;
}

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
  constexpr int G = D / 16;
  const Task k = find_task<D>(a);
  if (!k.block) return;
  const int lo = max(k.t0, k.half * 8), hi = min(k.t1, k.half * 8 + 8);
  if (lo >= hi) return;
  const bool values = blockIdx.y != 0;
  const E* base = static_cast<const E*>(values ? a.v : a.k);
  const long long* st = values ? a.vs : a.ks;
  base += k.b * st[0] + k.h * st[2] + k.g * 16;
  if (!values) {
    for (int t = lo; t < hi; ++t) {
      float x[16];
      uint32_t u[16];
      load_group(base + (k.first + t) * st[1], vec, x);
      const uint32_t byte = quantise(x, u);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) word |= kv_place(u[8 * w + e], e);
        *reinterpret_cast<uint32_t*>(k.block + k_word_offset<D>(t, 2 * k.g + w)) = word;
      }
      k.block[k_scale_offset<D>(t, k.g)] = static_cast<uint8_t>(byte);
    }
  } else {
    uint32_t word[16] = {}, keep = 0xFFFFFFFFu;
    for (int t = lo; t < hi; ++t) {
      float x[16];
      uint32_t u[16];
      load_group(base + (k.first + t) * st[1], vec, x);
      const uint32_t byte = quantise(x, u);
#pragma unroll
      for (int d = 0; d < 16; ++d) word[d] |= kv_place(u[d], t & 7);
      keep &= ~kv_place(15u, t & 7);
      k.block[kv_v_scales(D) + k.g * kKvBlock + t] = static_cast<uint8_t>(byte);
    }
#pragma unroll
    for (int d = 0; d < 16; ++d) {
      uint32_t* p = reinterpret_cast<uint32_t*>(k.block + v_word_offset<D>(k.g * 16 + d, k.half));
      *p = word[d] | (keep ? *p & keep : 0u);
    }
  }
}

template <typename E>
__device__ __forceinline__ void store_group(E* p, const float (&x)[16]) {
  if constexpr (sizeof(E) == 2) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}

// Rows past a request's count are zero; rows of a request in error are NaN.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvStoreArgs a) {
  constexpr int G = D / 16;
  const Task k = find_task<D>(a);
  if (k.b < 0) return;
  const bool values = blockIdx.y != 0;
  E* out = static_cast<E*>(values ? a.out_v : a.out_k) +
           (static_cast<long long>(k.b) * a.n * a.c.kv_heads + k.h) * D + k.g * 16;
  const long long row = static_cast<long long>(a.c.kv_heads) * D;
  uint32_t vw[16];
  if (values && k.block) {
#pragma unroll
    for (int d = 0; d < 16; ++d)
      vw[d] = *reinterpret_cast<const uint32_t*>(k.block + v_word_offset<D>(k.g * 16 + d, k.half));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = k.half * 8 + i;
    const long long at = k.first + t;
    if (at < 0 || at >= a.n) continue;
    float x[16];
    const bool live = t >= k.t0 && t < k.t1;
#pragma unroll
    for (int d = 0; d < 16; ++d) x[d] = k.bad && live ? __int_as_float(0x7FC00000) : 0.f;
    if (live && k.block) {
      if (!values) {
        const float s = kv_scale(k.block[k_scale_offset<D>(t, k.g)]);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t word = *reinterpret_cast<const uint32_t*>(k.block + k_word_offset<D>(t, 2 * k.g + w));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[8 * w + e] = kv_code(word, e) * s;
        }
      } else {
        const float s = kv_scale(k.block[kv_v_scales(D) + k.g * kKvBlock + t]);
#pragma unroll
        for (int d = 0; d < 16; ++d) x[d] = kv_code(vw[d], i) * s;
      }
    }
    store_group(out + at * row, x);
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
  if (D == 64) kv_read_kernel<E, 64><<<grid, kThreads, 0, s>>>(a);
  else if (D == 128) kv_read_kernel<E, 128><<<grid, kThreads, 0, s>>>(a);
  else kv_read_kernel<E, 256><<<grid, kThreads, 0, s>>>(a);
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
