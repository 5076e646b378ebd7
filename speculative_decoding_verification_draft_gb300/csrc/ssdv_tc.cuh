// ssdv_tc.cuh -- tensor memory, matrix instructions and bounded waits of the kernels
// on the fifth-generation tensor cores.
#pragma once

#include "ssdv_attn.cuh"

namespace ssdv {
namespace {

// ---- tcgen05 ----

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// (one lane's)
__device__ __forceinline__ void tc_commit(uint32_t bar, bool leader) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}
// 16 columns of the warp's 32 lanes; not to be used before tc_wait_ld.
__device__ __forceinline__ void tc_ld16(uint32_t at, float* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]),
        "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
      : "r"(at));
}
__device__ __forceinline__ void tc_ld8(uint32_t at, float* x) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "r"(at));
}
__device__ __forceinline__ void tc_ld4(uint32_t at, float* x) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
               : "r"(at));
}
__device__ __forceinline__ void tc_wait_ld4(float* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]));
}
__device__ __forceinline__ void tc_st4(uint32_t at, const float (&x)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3])
               : "memory");
}
// Waits for the loads; the registers pass through, so that no use moves ahead.
template <int N>
__device__ __forceinline__ void tc_wait_ld(float* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile(""
                 : "+f"(x[i]), "+f"(x[i + 1]), "+f"(x[i + 2]), "+f"(x[i + 3]), "+f"(x[i + 4]), "+f"(x[i + 5]),
                   "+f"(x[i + 6]), "+f"(x[i + 7]));
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t at, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// D [128 x N] in tensor memory (+)= A [128 x 16] in tensor memory, B [N x 16] in shared memory.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, bool leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(leader))
      : "memory");
}
// fp16 x fp16 -> fp32, M = 128, A contraction-major; B so (rows of 64 of the
// contraction) or row-major (64 rows at each of the contraction).
__device__ __forceinline__ constexpr uint32_t tc_idesc(int n, bool row_major) {
  return (1u << 4) | (row_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) | ((128u / 16) << 24);
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
template <int kCount = 128>
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kCount) : "memory");
}
template <int kCount>
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "bar.red.or.pred p, %1, %3, q;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(x)), "n"(kCount)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float lds_f(uint32_t p) { return __uint_as_float(lds32(p)); }
__device__ __forceinline__ void sts_f(uint32_t p, float x) { sts32(p, __float_as_uint(x)); }
__device__ __forceinline__ int warp_of(int tid) { return tid >> 5; }
__device__ __forceinline__ void sts16(uint32_t p, uint32_t x) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(p), "h"(static_cast<unsigned short>(x)) : "memory");
}
__device__ __forceinline__ uint32_t lds16(uint32_t p) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p));
  return v;
}
// (x, y) = (x, y) * (f.x, f.y) + (f.z, f.w), and (x, y) += (a, b): two fp32 operations at once.
__device__ __forceinline__ void fma_pair(float& x, float& y, const uint4& f) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "r"(f.x), "r"(f.y), "r"(f.z), "r"(f.w));
}
__device__ __forceinline__ void add_pair(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// Sums over lanes of kRows rows; the rows that a lane ends with begin at the row
// returned.  Rows are exchanged, so that each step halves what a lane holds.
template <int kRows, int kBit, int kMost>
__device__ __forceinline__ int lane_sums(float (&l)[kMost], int lane) {
  if constexpr (kBit == 0) {
    return 0;
  } else if constexpr (kRows % 2 == 0) {
    constexpr int kHalf = kRows / 2;
    const bool upper = lane & kBit;
#pragma unroll
    for (int n = 0; n < kHalf; ++n) {
      const float mine = upper ? l[n + kHalf] : l[n], other = upper ? l[n] : l[n + kHalf];
      l[n] = mine + __shfl_xor_sync(~0u, other, kBit);
    }
    return (upper ? kHalf : 0) + lane_sums<kHalf, kBit / 2>(l, lane);
  } else {
#pragma unroll
    for (int n = 0; n < kRows; ++n) l[n] += __shfl_xor_sync(~0u, l[n], kBit);
    return lane_sums<kRows, kBit / 2>(l, lane);
  }
}

// Waits that end: once one has run out, the warp goes through the motions
// without waiting, so that every barrier of the CTA is still met.
struct Waiter {
  uint32_t bars;
  int tries = 1 << 24;  // of about a hundred cycles; zero once a wait has run out
  __device__ __forceinline__ bool dead() const { return tries == 0; }
  // (as short as it gets: there are many of them, and instruction fetches are scarce)
  __device__ __forceinline__ void wait(int bar, uint32_t phase) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 n;\n\tmov.b32 n, %0;\n"
        "TRY:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "sub.s32 n, n, 1;\n\tsetp.gt.s32 p, n, 0;\n\t@p bra TRY;\n\tmov.b32 %0, 0;\nDONE:\n\t}"
        : "+r"(tries)
        : "r"(bars + bar * 8), "r"(phase & 1)
        : "memory");
  }
  // For warps that run ahead: they sleep between tries.
  __device__ __forceinline__ void nap(int bar, uint32_t phase) {
#pragma unroll 1
    for (int i = 0; i < (1 << 22) && !dead(); ++i) {
      if (bar_test(bars + bar * 8, phase & 1)) return;
      __nanosleep(200);
    }
    tries = 0;
  }
  __device__ __forceinline__ void arrive(int bar) { bar_arrive(bars + bar * 8); }
};

}  // namespace
}  // namespace ssdv
