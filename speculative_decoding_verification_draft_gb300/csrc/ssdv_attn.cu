// ssdv_attn.cu -- attention of a round's query tokens over the 4-bit cache.
//
// Query i of request b sits at position L_b + i and sees the positions
// [lo, hi): hi = L_b + i + 1 (its own key included), or L_b with past_only;
// lo = max(0, L_b + i + 1 - window) if there is a window, else 0.
//   out = sum_p exp(c q.k_p) v_p / sum_p exp(c q.k_p),  lse = log of that sum
// with the running maximum and sum of the softmax in 32 bits.  A row that sees
// nothing has out = 0 and lse = -inf.
#include "ssdv_kv.cuh"

namespace ssdv {

namespace {

constexpr int kThreads = 128;

// One CTA per (query row, kv head, request): a thread scores one token of a
// 128-token tile, then holds one (D = 256: two) of the output's elements.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) kv_attention_kernel(KvAttnArgs a) {
  constexpr int G = D / 16;
  constexpr int kPer = D > kThreads ? D / kThreads : 1;
  __shared__ float sq[D], sp[kThreads], red[4];
  __shared__ long long sblk[kThreads / kKvBlock];
  const int per_kv = a.heads / a.c.kv_heads;
  const int b = blockIdx.z, h = blockIdx.y, i = blockIdx.x / per_kv, head = h * per_kv + blockIdx.x % per_kv;
  const int tid = threadIdx.x;
  const int len = a.kv_len[b], nq = a.n_q ? a.n_q[b] : a.nq;
  const long long orow = (static_cast<long long>(b) * a.nq + i) * a.heads + head;
  E* out = static_cast<E*>(a.out) + orow * D;
  bool bad = len < 0 || nq < 0 || nq > a.nq ||
             static_cast<long long>(len) + (a.past_only ? 0 : nq) > static_cast<long long>(a.c.max_pages) * a.c.page_size;
  if (bad && tid == 0 && blockIdx.x == 0 && h == 0) atomicOr(a.status, 1 << SSD_ERR_LENGTH);
  int hi = 0, lo = 0;
  if (!bad && i < nq) {
    hi = a.past_only ? len : len + i + 1;
    lo = a.window ? max(0, len + i + 1 - a.window) : 0;
  }
  for (int d = tid; d < D; d += kThreads)
    sq[d] = static_cast<float>(static_cast<const E*>(a.q)[b * a.qs[0] + i * a.qs[1] + head * a.qs[2] + d]);
  float m = -INFINITY, l = 0.f, acc[kPer] = {};
  const int per_page = a.c.page_size / kKvBlock;
  for (int t0 = lo / kThreads * kThreads; t0 < hi; t0 += kThreads) {
    __syncthreads();
    if (tid < kThreads / kKvBlock) {
      const int pos = t0 + tid * kKvBlock;
      long long at = -2;  // not visited
      if (pos < hi && pos + kKvBlock > lo) {
        const int page = a.c.page_table[static_cast<long long>(b) * a.c.max_pages + pos / a.c.page_size];
        at = page < 0 || page >= a.c.n_pages
                 ? -1
                 : (static_cast<long long>(page) * a.c.kv_heads + h) * per_page + pos / kKvBlock % per_page;
        if (at == -1) atomicOr(a.status, 1 << SSD_ERR_PAGE);
      }
      sblk[tid] = at;
    }
    __syncthreads();
    const int t = t0 + tid, s = tid % kKvBlock;
    const long long at = sblk[tid / kKvBlock];
    float score = -INFINITY;
    if (t >= lo && t < hi && at >= 0) {
      const uint8_t* blk = a.c.pages + at * kv_block_bytes(D);
      float dot = 0.f;
      for (int g = 0; g < G; ++g) {
        float part = 0.f;
        for (int w = 0; w < 2; ++w) {
          const uint32_t word = *reinterpret_cast<const uint32_t*>(blk + k_word_offset<D>(s, 2 * g + w));
          for (int e = 0; e < 8; ++e) part += sq[16 * g + 8 * w + e] * kv_code(word, e);
        }
        dot += part * kv_scale(blk[kv_k_scales(D) + s * G + g]);
      }
      score = dot * a.scale_log2;
    }
    for (int x = 0; x < kThreads / kKvBlock; ++x) bad |= sblk[x] == -1;
    // fmaxf drops a NaN score; it comes back through its weight
    float top = score;
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (tid % 32 == 0) red[tid / 32] = top;
    __syncthreads();
    top = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float ref = top == -INFINITY ? 0.f : top;
    const float p = exp2f(score - ref), old = exp2f(m - ref);
    sp[tid] = p;
    __syncthreads();
    float sum = 0.f;
    for (int x = 0; x < kThreads; ++x) sum += sp[x];
    l = l * old + sum;
    m = top;
    for (int j = 0; j < kPer; ++j) {
      const int d = tid + j * kThreads;
      if (d >= D) continue;
      float y = acc[j] * old;
      for (int x = max(lo - t0, 0); x < min(hi - t0, kThreads); ++x) {
        if (sblk[x / kKvBlock] < 0) continue;
        const uint8_t* blk = a.c.pages + sblk[x / kKvBlock] * kv_block_bytes(D);
        const int u = x % kKvBlock;
        const uint32_t word = *reinterpret_cast<const uint32_t*>(blk + v_word_offset<D>(d, u >> 3));
        y += sp[x] * (kv_code(word, u & 7) * kv_scale(blk[kv_v_scales(D) + d / 16 * kKvBlock + u]));
      }
      acc[j] = y;
    }
  }
  const float inv = bad ? __int_as_float(0x7FC00000) : hi > lo ? 1.f / l : 0.f;
  for (int j = 0; j < kPer; ++j)
    if (tid + j * kThreads < D) out[tid + j * kThreads] = static_cast<E>(hi > lo || bad ? acc[j] * inv : 0.f);
  if (a.lse && tid == 0)
    a.lse[orow] = bad ? inv : hi > lo ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <typename E>
cudaError_t attention_dim(const KvAttnArgs& a, int D, cudaStream_t s) {
  const dim3 grid(a.nq * (a.heads / a.c.kv_heads), a.c.kv_heads, a.B);
  if (D == 64) kv_attention_kernel<E, 64><<<grid, kThreads, 0, s>>>(a);
  else if (D == 128) kv_attention_kernel<E, 128><<<grid, kThreads, 0, s>>>(a);
  else kv_attention_kernel<E, 256><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv_attention_work_bytes(int rows, int D) { return 0; }

cudaError_t launch_kv_attention(const KvAttnArgs& a, int D, int esize, cudaStream_t stream) {
  return esize == 2 ? attention_dim<__nv_bfloat16>(a, D, stream) : attention_dim<float>(a, D, stream);
}

}  // namespace ssdv
