// ple_kv_append / ple_kv_read: rows into and out of the paged 4-bit cache.
//
// Append: a row of head_dim elements belongs to head_dim / 8 neighbouring
// threads, eight elements (one 16-byte vector) each. A rotation pair of the
// half-split form lies rotary_dim / 16 threads apart, so partners are
// exchanged by shuffle; an interleaved pair lies in one thread. The row's
// minimum and maximum are a butterfly over the row's threads, and eight
// codes are one 32-bit word: every load and store is as wide as the row
// allows and each byte moves once. Bound by memory for large steps, by
// latency for small ones.
#include "kv_cache.cuh"

namespace ple {
namespace {

constexpr int kAppendThreads = 256;

struct AppendArgs {
  const ple_bf16_t* q;
  const ple_bf16_t* k;
  const ple_bf16_t* v;
  ple_bf16_t* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int64_t T;
  int num_heads;  // query heads (0: none)
  const float* cos_sin;
  int64_t num_positions;
  int rot;
  bool interleaved;
  const int32_t* positions;
  int32_t* dev_err;
};

// NaN if either is (fminf and fmaxf drop NaN).
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const AppendArgs a, const KvCache c) {
  constexpr int kLanes = D / 8;  // threads of a row
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  const int row = (blockIdx.y * kAppendThreads + threadIdx.x) / kLanes;
  const int e = threadIdx.x % kLanes;
  const int rows = a.num_heads + 2 * c.num_kv_heads;
  if (blockIdx.y == 0)
    for (int64_t i = t * kAppendThreads + threadIdx.x; i < c.num_reqs; i += int64_t(gridDim.x) * kAppendThreads)
      check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
  const int r = request_of(c.qsl, c.num_reqs, t);
  // rows past the last stay in the warp for the shuffles
  const bool live = row < rows;
  const bool is_q = row < a.num_heads;
  const bool is_v = row >= a.num_heads + c.num_kv_heads;
  const int h = is_q ? row : is_v ? row - a.num_heads - c.num_kv_heads : row - a.num_heads;

  int64_t p = -1;
  bool bad = false;  // a position outside the rotation table or the cache
  int64_t at = 0;
  if (r >= 0) {
    p = static_cast<int64_t>(__ldg(c.kv_lens + r)) - (static_cast<int64_t>(__ldg(c.qsl + r + 1)) - t);
    at = a.positions != nullptr ? __ldg(a.positions + t) : p;
    bad = a.cos_sin != nullptr && (at < 0 || at >= a.num_positions);
  }
  uint8_t* block = nullptr;
  if (r >= 0 && !bad && live && !is_q) {
    block = kv_block<D>(c, r, p, h);
    bad = block == nullptr;
  }
  if (bad) set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);

  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live && r >= 0 && !bad) {
    const ple_bf16_t* src = is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride;
    unpack8(*reinterpret_cast<const uint4*>(src + static_cast<int64_t>(h) * D + e * 8), x);
  }
  // The products and their sum are rounded one by one, so that a code does
  // not depend on how a compiler contracts them.
  if (a.cos_sin != nullptr) {
    const int half = a.rot / 2;
    const bool turn = live && !is_v && r >= 0 && !bad && e * 8 < a.rot;
    const float* cs = a.cos_sin + (turn ? at * a.rot : 0);
    if (a.interleaved) {
      if (turn) {
        const float4 co = __ldg(reinterpret_cast<const float4*>(cs + e * 4));
        const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + e * 4));
        const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = x[2 * i], w = x[2 * i + 1];
          x[2 * i] = __fsub_rn(__fmul_rn(u, cv[i]), __fmul_rn(w, sv[i]));
          x[2 * i + 1] = __fadd_rn(__fmul_rn(w, cv[i]), __fmul_rn(u, sv[i]));
        }
      }
    } else {
      const int lanes = half / 8;  // distance of a pair in threads
      const bool first = e < lanes;
      const int base = (threadIdx.x & 31) - e;
      const int partner = e * 8 < a.rot ? base + (first ? e + lanes : e - lanes) : base + e;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
      if (turn) {
        const int j = (first ? e : e - lanes) * 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 co = __ldg(reinterpret_cast<const float4*>(cs + j + i));
          const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + j + i));
          const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float m = __fmul_rn(x[i + n], cv[n]), o = __fmul_rn(y[i + n], sv[n]);
            x[i + n] = first ? __fsub_rn(m, o) : __fadd_rn(m, o);
          }
        }
      }
    }
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) { lo = min_nan(lo, x[i]); hi = max_nan(hi, x[i]); }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!live) return;
  if (is_q) {
    uint4 o;
    o.x = pack2(x[0], x[1]); o.y = pack2(x[2], x[3]); o.z = pack2(x[4], x[5]); o.w = pack2(x[6], x[7]);
    *reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + static_cast<int64_t>(h) * D + e * 8) = o;
    return;
  }
  if (block == nullptr) return;
  const uint32_t pair = pack2(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f), lo);  // (scale, offset)
  const float scale = bf_lo(pair), offset = bf_hi(pair);
  uint32_t word = 0;
  if (scale > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = rintf(__fdiv_rn(__fsub_rn(x[i], offset), scale));
      word |= static_cast<uint32_t>(fminf(fmaxf(y, 0.0f), 15.0f)) << (4 * i);
    }
  }
  const int slot = static_cast<int>(p % kBlockTokens);
  *reinterpret_cast<uint32_t*>(block + (is_v ? KvBlock<D>::kV : 0) + slot * KvBlock<D>::kRow + e * 4) = word;
  if (e == 0)
    *reinterpret_cast<uint32_t*>(block + (is_v ? KvBlock<D>::kVPairs : KvBlock<D>::kPairs) + slot * 4) = pair;
}

struct ReadArgs {
  ple_bf16_t* k_out;
  ple_bf16_t* v_out;
  int64_t T;
  int32_t* dev_err;
};

template <int D>
__global__ void __launch_bounds__(kAppendThreads)
kv_read_kernel(const ReadArgs a, const KvCache c) {
  constexpr int kLanes = D / 8;
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  const int row = (blockIdx.y * kAppendThreads + threadIdx.x) / kLanes;  // K heads, then V heads
  const int e = threadIdx.x % kLanes;
  if (blockIdx.y == 0)
    for (int64_t i = t * kAppendThreads + threadIdx.x; i < c.num_reqs; i += int64_t(gridDim.x) * kAppendThreads)
      check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
  const int r = request_of(c.qsl, c.num_reqs, t);
  if (row >= 2 * c.num_kv_heads) return;
  const bool is_v = row >= c.num_kv_heads;
  const int h = is_v ? row - c.num_kv_heads : row;
  ple_bf16_t* out = is_v ? a.v_out : a.k_out;
  if (out == nullptr) return;
  uint4 o = make_uint4(0, 0, 0, 0);
  if (r >= 0) {
    const int64_t p = static_cast<int64_t>(__ldg(c.kv_lens + r)) - (static_cast<int64_t>(__ldg(c.qsl + r + 1)) - t);
    const uint8_t* block = kv_block<D>(c, r, p, h);
    if (block == nullptr) {
      set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
    } else {
      const int slot = static_cast<int>(p % kBlockTokens);
      const uint32_t word = *reinterpret_cast<const uint32_t*>(
          block + (is_v ? KvBlock<D>::kV : 0) + slot * KvBlock<D>::kRow + e * 4);
      const uint32_t pair = *reinterpret_cast<const uint32_t*>(
          block + (is_v ? KvBlock<D>::kVPairs : KvBlock<D>::kPairs) + slot * 4);
      const float scale = bf_lo(pair), offset = bf_hi(pair);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = fmaf(static_cast<float>((word >> (4 * i)) & 15u), scale, offset);
      o.x = pack2(x[0], x[1]); o.y = pack2(x[2], x[3]); o.z = pack2(x[4], x[5]); o.w = pack2(x[6], x[7]);
    }
  }
  *reinterpret_cast<uint4*>(out + (t * c.num_kv_heads + h) * D + e * 8) = o;
}

dim3 row_grid(int64_t T, int rows, int D) {
  return dim3(static_cast<unsigned>(T), (rows * (D / 8) + kAppendThreads - 1) / kAppendThreads);
}

}  // namespace
}  // namespace ple

using namespace ple;

PLE_EXPORT size_t ple_kv_block_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 || head_dim == 256 ? size_t(kBlockTokens) * (head_dim + 8) : 0;
}

PLE_EXPORT ple_status ple_kv_append(const ple_bf16_t* q, int64_t q_stride, const ple_bf16_t* k,
                                    int64_t k_stride, const ple_bf16_t* v, int64_t v_stride,
                                    int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                                    int32_t head_dim, const float* cos_sin, int64_t num_positions,
                                    int32_t rotary_dim, int32_t interleaved,
                                    const int32_t* positions, void* cache, int64_t num_pages,
                                    int32_t page_size, const int32_t* block_table,
                                    int32_t max_pages, const int32_t* query_start_loc,
                                    int32_t num_reqs, const int32_t* kv_lens, ple_bf16_t* q_out,
                                    int64_t q_out_stride, int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_kv_append";
  if (num_tokens < 0 || num_tokens > INT32_MAX)
    return fail(PLE_ERR_INVALID_ARG, "%s: num_tokens %lld", name, static_cast<long long>(num_tokens));
  if (num_tokens == 0) return PLE_OK;
  if (ple_status s = check_cache(name, cache, num_pages, page_size, block_table, max_pages,
                                 query_start_loc, num_reqs, kv_lens, num_kv_heads, head_dim))
    return s;
  if (k == nullptr || v == nullptr || (q == nullptr) != (q_out == nullptr))
    return fail(PLE_ERR_INVALID_ARG, "%s: null k or v, or only one of q and q_out", name);
  if (q == nullptr) num_heads = 0;
  if (num_heads < (q != nullptr ? 1 : 0))
    return fail(PLE_ERR_INVALID_ARG, "%s: num_heads %d", name, num_heads);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(cos_sin))
    return fail(PLE_ERR_INVALID_ARG, "%s: q, k, v, q_out and cos_sin must be 16-byte aligned", name);
  if ((q != nullptr && (q_stride % 8 != 0 || q_out_stride % 8 != 0)) || k_stride % 8 != 0 || v_stride % 8 != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: row strides must be multiples of 8", name);
  if (cos_sin != nullptr && (rotary_dim <= 0 || rotary_dim % 16 != 0 || rotary_dim > head_dim))
    return fail(PLE_ERR_UNSUPPORTED, "%s: rotary_dim %d (a multiple of 16, at most head_dim)", name, rotary_dim);
  if (cos_sin != nullptr && num_positions < 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: num_positions %lld", name, static_cast<long long>(num_positions));
  const AppendArgs a{q, k, v, q_out, q_stride, k_stride, v_stride, q_out_stride, num_tokens, num_heads,
                     cos_sin, num_positions, cos_sin != nullptr ? rotary_dim : 0, interleaved != 0,
                     positions, dev_err};
  const KvCache c{static_cast<uint8_t*>(cache), num_pages, page_size, num_kv_heads, block_table,
                  max_pages, query_start_loc, num_reqs, kv_lens};
  const dim3 grid = row_grid(num_tokens, num_heads + 2 * num_kv_heads, head_dim);
  const auto kernel = head_dim == 64 ? kv_append_kernel<64> : head_dim == 128 ? kv_append_kernel<128> : kv_append_kernel<256>;
  return check_cuda(launch_kernel(kernel, grid, dim3(kAppendThreads), 0, stream, 1, a, c), name);
}

PLE_EXPORT ple_status ple_kv_read(const void* cache, int64_t num_pages, int32_t page_size,
                                  const int32_t* block_table, int32_t max_pages,
                                  const int32_t* query_start_loc, int32_t num_reqs,
                                  const int32_t* kv_lens, int64_t num_tokens, int32_t num_kv_heads,
                                  int32_t head_dim, ple_bf16_t* k_out, ple_bf16_t* v_out,
                                  int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_kv_read";
  if (num_tokens < 0 || num_tokens > INT32_MAX)
    return fail(PLE_ERR_INVALID_ARG, "%s: num_tokens %lld", name, static_cast<long long>(num_tokens));
  if (num_tokens == 0 || (k_out == nullptr && v_out == nullptr)) return PLE_OK;
  if (ple_status s = check_cache(name, cache, num_pages, page_size, block_table, max_pages,
                                 query_start_loc, num_reqs, kv_lens, num_kv_heads, head_dim))
    return s;
  if (!aligned16(k_out) || !aligned16(v_out))
    return fail(PLE_ERR_INVALID_ARG, "%s: k_out and v_out must be 16-byte aligned", name);
  const ReadArgs a{k_out, v_out, num_tokens, dev_err};
  const KvCache c{const_cast<uint8_t*>(static_cast<const uint8_t*>(cache)), num_pages, page_size,
                  num_kv_heads, block_table, max_pages, query_start_loc, num_reqs, kv_lens};
  const dim3 grid = row_grid(num_tokens, 2 * num_kv_heads, head_dim);
  const auto kernel = head_dim == 64 ? kv_read_kernel<64> : head_dim == 128 ? kv_read_kernel<128> : kv_read_kernel<256>;
  return check_cuda(launch_kernel(kernel, grid, dim3(kAppendThreads), 0, stream, 1, a, c), name);
}
