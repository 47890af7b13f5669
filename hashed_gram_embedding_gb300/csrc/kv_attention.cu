// ple_kv_attention: grouped-query attention over the paged 4-bit cache.
//
// One warp per (token, query head). Scores are taken 32 positions at a time,
// one position per lane; with a running maximum m and sum l the softmax
// needs one pass: o and l are scaled by exp(m_old - m_new) when m grows.
#include "kv_cache.cuh"

#include <cmath>

namespace ple {
namespace {

constexpr int kThreads = 128;

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
};

template <int D>
__global__ void __launch_bounds__(kThreads)
attention_rows_kernel(const AttentionArgs a, const KvCache c) {
  constexpr int kPer = D / 32;  // output elements of a lane
  __shared__ float qs[kThreads / 32][D];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t row = int64_t(blockIdx.x) * (kThreads / 32) + warp;
  if (row >= a.T * a.num_heads) return;
  const int64_t t = row / a.num_heads;
  const int h = static_cast<int>(row % a.num_heads);
  const int hk = h / (a.num_heads / c.num_kv_heads);
  if (h == 0)
    for (int64_t i = t * 32 + lane; i < c.num_reqs; i += a.T * 32) check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
  for (int i = lane; i < D; i += 32) qs[warp][i] = bf_lo(a.q[t * a.q_stride + int64_t(h) * D + i]);
  __syncwarp();
  float o[kPer] = {};
  float m = -INFINITY, l = 0.0f;
  const int r = request_of(c.qsl, c.num_reqs, t);
  if (r >= 0) {
    const int64_t len = __ldg(c.kv_lens + r);
    const int64_t last = a.causal ? len - (__ldg(c.qsl + r + 1) - t) : len - 1;
    const int64_t first = a.window > 0 && last - a.window + 1 > 0 ? last - a.window + 1 : 0;
    for (int64_t p0 = first; p0 <= last; p0 += 32) {
      const int64_t p = p0 + lane;
      float s = -INFINITY;
      const uint8_t* block = p <= last ? kv_block<D>(c, r, p, hk) : nullptr;
      if (p <= last && block == nullptr) set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
      const int slot = static_cast<int>(p % kBlockTokens);
      uint32_t vpair = 0;
      if (block != nullptr) {
        const uint32_t pair = *reinterpret_cast<const uint32_t*>(block + KvBlock<D>::kPairs + slot * 4);
        vpair = *reinterpret_cast<const uint32_t*>(block + KvBlock<D>::kVPairs + slot * 4);
        const uint32_t* k = reinterpret_cast<const uint32_t*>(block + slot * KvBlock<D>::kRow);
        s = 0.0f;
        for (int w = 0; w < D / 8; ++w) {
          const uint32_t word = k[w];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            s = fmaf(qs[warp][w * 8 + i], fmaf(static_cast<float>((word >> (4 * i)) & 15u), bf_lo(pair), bf_hi(pair)), s);
        }
        s *= a.scale_log2;
      }
      float top = s;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float next = fmaxf(m, top);
      const float base = next == -INFINITY ? 0.0f : next;
      const float keep = exp2f(m - base);
      const float w = block != nullptr ? exp2f(s - base) : 0.0f;
      l = l * keep + warp_sum(w);
      m = next;
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[i] *= keep;
      for (int i = 0; i < 32; ++i) {
        const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(block), i);
        if (at == 0) continue;
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const uint32_t pair = __shfl_sync(0xffffffffu, vpair, i);
        const uint8_t* v = reinterpret_cast<const uint8_t*>(at) + KvBlock<D>::kV +
                           static_cast<int>((p0 + i) % kBlockTokens) * KvBlock<D>::kRow;
#pragma unroll
        for (int n = 0; n < kPer; n += 2) {
          const uint32_t b = v[lane * (kPer / 2) + n / 2];
          o[n] = fmaf(wi, fmaf(static_cast<float>(b & 15u), bf_lo(pair), bf_hi(pair)), o[n]);
          o[n + 1] = fmaf(wi, fmaf(static_cast<float>(b >> 4), bf_lo(pair), bf_hi(pair)), o[n + 1]);
        }
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  ple_bf16_t* dst = a.out + t * a.out_stride + int64_t(h) * D + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack2(o[i] * inv, o[i + 1] * inv);
}

}  // namespace
}  // namespace ple

using namespace ple;

PLE_EXPORT size_t ple_kv_attention_workspace(int32_t num_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 || ple_kv_block_bytes(head_dim) == 0)
    return 0;
  return 256;
}

PLE_EXPORT ple_status ple_kv_attention(const ple_bf16_t* q, int64_t q_stride, int64_t num_tokens,
                                       int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                       const void* cache, int64_t num_pages, int32_t page_size,
                                       const int32_t* block_table, int32_t max_pages,
                                       const int32_t* query_start_loc, int32_t num_reqs,
                                       const int32_t* kv_lens, int32_t max_query_len, float scale,
                                       int32_t causal, int32_t window, ple_bf16_t* out,
                                       int64_t out_stride, void* workspace, size_t workspace_bytes,
                                       int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_kv_attention";
  if (num_tokens < 0 || num_tokens > INT32_MAX)
    return fail(PLE_ERR_INVALID_ARG, "%s: num_tokens %lld", name, static_cast<long long>(num_tokens));
  if (num_tokens == 0) return PLE_OK;
  if (ple_status s = check_cache(name, cache, num_pages, page_size, block_table, max_pages,
                                 query_start_loc, num_reqs, kv_lens, num_kv_heads, head_dim))
    return s;
  if (num_heads < 1 || num_heads % num_kv_heads != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: %d heads over %d kv heads", name, num_heads, num_kv_heads);
  if (q == nullptr || out == nullptr || !aligned16(q) || !aligned16(out) || q_stride % 8 != 0 || out_stride % 8 != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned, their strides multiples of 8", name);
  if (!(scale > 0.0f) || !std::isfinite(scale))
    return fail(PLE_ERR_INVALID_ARG, "%s: scale %g", name, scale);
  if (max_query_len < 0 || window < 0 || (window > 0 && !causal))
    return fail(PLE_ERR_INVALID_ARG, "%s: max_query_len %d, window %d%s", name, max_query_len, window,
                causal ? "" : " without causal");
  const size_t need = ple_kv_attention_workspace(num_heads, num_kv_heads, head_dim);
  if (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: workspace of %zu bytes, 256-byte aligned, needed", name, need);
  const AttentionArgs a{q, q_stride, num_tokens, num_heads, scale * 1.4426950408889634f, causal != 0,
                        window, out, out_stride, dev_err};
  const KvCache c{const_cast<uint8_t*>(static_cast<const uint8_t*>(cache)), num_pages, page_size,
                  num_kv_heads, block_table, max_pages, query_start_loc, num_reqs, kv_lens};
  const int64_t rows = num_tokens * num_heads;
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
  const auto kernel = head_dim == 64 ? attention_rows_kernel<64> : head_dim == 128 ? attention_rows_kernel<128>
                                                                                  : attention_rows_kernel<256>;
  return check_cuda(launch_kernel(kernel, grid, dim3(kThreads), 0, stream, 1, a, c), name);
}
