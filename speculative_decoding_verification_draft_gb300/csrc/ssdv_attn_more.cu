// ssdv_attn_more.cu -- the kernels of ssdv_attn.cu with sinks, first positions and
// sums in place of outputs (ssdv_attn.cuh says why they stand apart).
#define SSDV_ATTN_MORE 1
#include "ssdv_attn.cu"
