// What the two kernels of ple_kv_attention share: one for requests of few
// query rows (kv_attention.cu), one for requests of many (kv_prefill.cu).
#pragma once

#include "codes.cuh"
#include "kv_cache.cuh"

namespace ple {

struct AttentionArgs {
  const ple_bf16_t* q;
  int64_t q_stride;
  int64_t T;
  int num_heads;
  float scale_log2;  // scale * log2(e)
  bool causal;
  int window;
  ple_bf16_t* out;
  int64_t out_stride;
  int32_t* dev_err;
  int many_rows;     // requests with this many query rows a kv head or more go to the second kernel
};

// Attention of the requests with many rows. room:
// device memory for the results of shared rows, 256-byte aligned, of any content.
cudaError_t launch_prefill(const AttentionArgs& a, const KvCache& c, int head_dim, void* room, size_t room_bytes,
                           cudaStream_t stream);

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace ple
