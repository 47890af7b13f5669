// ple_proj_w4: out = x W^T with W in 4 bits, a scale and a zero point per
// group of columns, for steps of few tokens.
//
// With c the codes, sum_e x_e s (c_e - z) over a group is
// s * (sum_e x_e c_e - z * sum_e x_e): the codes enter the products as they
// are and the scale meets the float32 sum once per group.
#include "common.cuh"

namespace ple {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
proj_w4_kernel(const ple_bf16_t* __restrict__ x, int64_t x_stride, int64_t T, int E, int N,
               const uint8_t* __restrict__ codes, const ple_bf16_t* __restrict__ scales,
               const uint8_t* __restrict__ zeros, int group, ple_bf16_t* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int n = (blockIdx.x * kThreads + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = int64_t(blockIdx.y) * 8;
  if (n >= N) return;
  const int groups = E / group;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int e = lane * 8; e < E; e += 256) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + int64_t(n) * (E / 2) + e / 2);
    const int g = e / group;
    const float s = bf_lo(scales[int64_t(n) * groups + g]);
    const float z = zeros != nullptr ? float(zeros[int64_t(n) * groups + g]) : 8.0f;
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s * (float((w >> (4 * i)) & 15u) - z);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t0 + t >= T) break;
      float f[8];
      unpack8(ldg16(x + (t0 + t) * x_stride + e), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t] = fmaf(c[i], f[i], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const float v = warp_sum(acc[t]);
    if (lane == 0 && t0 + t < T) out[(t0 + t) * N + n] = static_cast<ple_bf16_t>(pack2(v, 0.0f) & 0xffffu);
  }
}

}  // namespace
}  // namespace ple

using namespace ple;

PLE_EXPORT ple_status ple_proj_w4(const ple_bf16_t* x, int64_t x_stride, int64_t num_tokens,
                                  int32_t in_dim, int32_t out_dim, const uint8_t* codes,
                                  const ple_bf16_t* scales, const uint8_t* zeros, int32_t group,
                                  ple_bf16_t* out, int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_proj_w4";
  (void)dev_err;
  if (num_tokens < 0 || num_tokens > INT32_MAX || in_dim < 1 || out_dim < 1)
    return fail(PLE_ERR_INVALID_ARG, "%s: num_tokens %lld, in_dim %d, out_dim %d", name,
                static_cast<long long>(num_tokens), in_dim, out_dim);
  if (group != 32 && group != 64 && group != 128)
    return fail(PLE_ERR_UNSUPPORTED, "%s: group %d (32, 64 or 128)", name, group);
  if (in_dim % group != 0)
    return fail(PLE_ERR_UNSUPPORTED, "%s: in_dim %d is not a multiple of the group %d", name, in_dim, group);
  if (num_tokens == 0) return PLE_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr || out == nullptr)
    return fail(PLE_ERR_INVALID_ARG, "%s: null x, codes, scales or out", name);
  if (!aligned16(x) || !aligned16(codes) || x_stride % 8 != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: x and codes must be 16-byte aligned, x_stride a multiple of 8", name);
  const dim3 grid((out_dim + 7) / 8, static_cast<unsigned>((num_tokens + 7) / 8));
  return check_cuda(launch_kernel(proj_w4_kernel, grid, dim3(kThreads), 0, stream, 1, x, x_stride,
                                  num_tokens, in_dim, out_dim, codes, scales, zeros, group, out), name);
}
