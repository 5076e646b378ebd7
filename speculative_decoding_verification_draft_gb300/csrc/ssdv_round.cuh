// ssdv_round.cuh -- launch arguments of what a round needs around the cache
// (ssdv_plan.cu: page tables and slots; ssdv_rope.cu: norms and rotation of
// queries and keys).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssdv {

struct KvPlanArgs {
  const int32_t* table;   // [B, max_pages]
  const int32_t* held;    // [B]
  const int32_t* free;    // [n_pages]
  const int32_t* n_free;  // [1]
  const int32_t* len;     // [B]
  const int32_t* n_new;   // [B] or null (n each)
  const int32_t* shared;  // [B] or null (none)
  int B, max_pages, n_pages, page_size, n;
  int32_t* out_table;
  int32_t* out_held;
  int32_t* out_free;
  int32_t* out_n_free;
  int64_t* slots;         // [B, n] or null
  int32_t* status;
  int4* work;             // [1 + B]
};
cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream);

struct RopeArgs {
  const void* q;
  const void* k;
  void* out_q;
  void* out_k;
  long long qs[3], ks[3], oqs[3], oks[3];  // element strides of request, token, head
  const int32_t* len;
  const int32_t* n_new;
  int B, n, heads, kv_heads;
  const float* q_weight;  // [D] or null: no norm
  const float* k_weight;
  const float* freq;      // [rot / 2]
  float eps;
  int rot;
  int32_t* status;
};
cudaError_t launch_rope(const RopeArgs& a, int D, int esize, bool interleaved, bool vec, cudaStream_t stream);

}  // namespace ssdv
