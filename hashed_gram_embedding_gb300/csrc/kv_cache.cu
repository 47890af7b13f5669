// ple_kv_append / ple_kv_read: rows into and out of the paged 4-bit cache.
//
// A row of head_dim elements belongs to head_dim / 8 neighbouring lanes, eight
// elements (one 16-byte vector) each, so every load and store is as wide as
// the row allows and each byte moves once. A rotation pair of the half-split
// form lies rotary_dim / 16 lanes apart, so partners are exchanged by shuffle;
// an interleaved pair lies in one lane. The row's minimum and maximum are a
// butterfly over its lanes, and eight codes are one 32-bit word.
//
// A warp looks its token up once - request, position, page, rotation - and
// then takes rows of it in turn: all of them when there are tokens enough to
// fill the card, one when there are few and latency counts. Bound by memory
// for large steps and by latency for small ones, as long as a row costs few
// instructions (a warp for each two rows of a token, with a division for each
// element, took 93 us where this takes the time stated at the launch).
#include "kv_cache.cuh"

namespace ple {
namespace {

constexpr int kAppendThreads = 128;

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

// Where a token lies. r: its request, -1 for padding; block: its block of kv
// head 0 (heads are head_stride bytes apart), nullptr outside the cache.
struct Place {
  int r;
  int64_t p;
  uint8_t* block;
  int64_t head_stride;
  int slot;
};

template <int D>
__device__ __forceinline__ Place place_of(const KvCache& c, int64_t t) {
  Place x;
  x.r = request_of(c.qsl, c.num_reqs, t);
  x.p = -1;
  x.block = nullptr;
  x.slot = 0;
  x.head_stride = static_cast<int64_t>(c.page_size / kBlockTokens) * KvBlock<D>::kBytes;
  if (x.r >= 0) {
    x.p = static_cast<int64_t>(__ldg(c.kv_lens + x.r)) - (static_cast<int64_t>(__ldg(c.qsl + x.r + 1)) - t);
    x.block = kv_block<D>(c, x.r, x.p, 0);
    x.slot = static_cast<int>(x.p & (kBlockTokens - 1));
  }
  return x;
}

// clamp(rint(y / scale), 0, 15) for eight values y = x - offset, packed. The
// quotient is taken as a product with the reciprocal, within 2^-22 of it
// relative, and rounded by adding 1.5 * 2^23; where it comes near a half, the
// division decides.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float scale, float offset) {
  constexpr float kRound = 12582912.0f;
  uint32_t word = 0;
  const float inv = __frcp_rn(scale);
  bool near = !(scale >= 1e-37f && scale <= 1e37f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], offset), inv), 0.0f), 15.0f);
    const float up = __fadd_rn(q, kRound);
    near |= fabsf(__fsub_rn(q, __fsub_rn(up, kRound))) > 0.4999f;
    word += (__float_as_uint(up) & 15u) << (4 * i);
  }
  if (near) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = rintf(__fdiv_rn(__fsub_rn(x[i], offset), scale));
      word |= static_cast<uint32_t>(fminf(fmaxf(y, 0.0f), 15.0f)) << (4 * i);
    }
  }
  return word;
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const AppendArgs a, const KvCache c) {
  constexpr int kLanes = D / 8;          // lanes of a row
  constexpr int kAtOnce = 32 / kLanes;   // rows of a warp
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int e = lane % kLanes;
  const int rows = a.num_heads + 2 * c.num_kv_heads;
  const int stride = gridDim.y * (kAppendThreads / 32) * kAtOnce;
  int row = (blockIdx.y * (kAppendThreads / 32) + threadIdx.x / 32) * kAtOnce + lane / kLanes;
  auto load = [&](int row) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const bool is_q = row < a.num_heads, is_v = row >= a.num_heads + c.num_kv_heads;
      const int h = is_q ? row : is_v ? row - a.num_heads - c.num_kv_heads : row - a.num_heads;
      const ple_bf16_t* src = is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride;
      v = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(h) * D + e * 8);
    }
    return v;
  };
  uint4 raw = load(row);  // on its way while the token is looked up
  if (blockIdx.y == 0)
    for (int64_t i = t * kAppendThreads + threadIdx.x; i < c.num_reqs; i += int64_t(gridDim.x) * kAppendThreads)
      check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
  const Place at = place_of<D>(c, t);
  bool none = at.r < 0;  // nothing to store, zeros for the query
  int64_t angle = 0;
  if (!none) {
    angle = a.positions != nullptr ? __ldg(a.positions + t) : at.p;
    const bool outside = a.cos_sin != nullptr && (angle < 0 || angle >= a.num_positions);
    if ((outside || at.block == nullptr) && lane == 0) set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
    none = outside;
  }
  const bool turns = a.cos_sin != nullptr && !none && e * 8 < a.rot;
  const int half = a.rot / 2;
  const int apart = half / 8;        // lanes between the two of a pair
  const bool first = e < apart;
  float co[8], si[8];                // interleaved: of four pairs
  if (turns) {
    const float* cs = a.cos_sin + angle * a.rot;
    if (a.interleaved) {
      *reinterpret_cast<float4*>(co) = __ldg(reinterpret_cast<const float4*>(cs + e * 4));
      *reinterpret_cast<float4*>(si) = __ldg(reinterpret_cast<const float4*>(cs + half + e * 4));
    } else {
      const int j = (first ? e : e - apart) * 8;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(co + i) = __ldg(reinterpret_cast<const float4*>(cs + j + i));
        *reinterpret_cast<float4*>(si + i) = __ldg(reinterpret_cast<const float4*>(cs + half + j + i));
      }
    }
  }
  const int partner = lane - e + (!turns ? e : first ? e + apart : e - apart);
  // rows past the last stay in the warp for the shuffles
  for (; __any_sync(0xffffffffu, row < rows); row += stride) {
    const uint4 next = load(row + stride);
    const bool live = row < rows;
    const bool is_q = row < a.num_heads, is_v = row >= a.num_heads + c.num_kv_heads;
    float x[8];
    unpack8(raw, x);
    // The products and their sum are rounded one by one, so that a code does
    // not depend on how a compiler contracts them.
    if (a.cos_sin != nullptr && __any_sync(0xffffffffu, !is_v)) {
      if (a.interleaved) {
        if (turns && !is_v) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = x[2 * i], w = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(u, co[i]), __fmul_rn(w, si[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(w, co[i]), __fmul_rn(u, si[i]));
          }
        }
      } else {
        uint4 other;
        other.x = __shfl_sync(0xffffffffu, raw.x, partner);
        other.y = __shfl_sync(0xffffffffu, raw.y, partner);
        other.z = __shfl_sync(0xffffffffu, raw.z, partner);
        other.w = __shfl_sync(0xffffffffu, raw.w, partner);
        if (turns && !is_v) {
          float y[8];
          unpack8(other, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float m = __fmul_rn(x[i], co[i]), o = __fmul_rn(y[i], si[i]);
            x[i] = first ? __fsub_rn(m, o) : __fadd_rn(m, o);
          }
        }
      }
    }
    raw = next;
    if (__any_sync(0xffffffffu, live && !is_q)) {
      float lo = x[0], hi = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) { lo = min_nan(lo, x[i]); hi = max_nan(hi, x[i]); }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      if (live && !is_q && !none && at.block != nullptr) {
        const int h = is_v ? row - a.num_heads - c.num_kv_heads : row - a.num_heads;
        uint8_t* block = at.block + h * at.head_stride;
        const uint32_t pair = pack2(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f), lo);  // (scale, offset)
        const float scale = bf_lo(pair);
        const uint32_t word = scale > 0.0f ? codes_of(x, scale, bf_hi(pair)) : 0u;
        *reinterpret_cast<uint32_t*>(block + (is_v ? KvBlock<D>::kV : 0) + at.slot * KvBlock<D>::kRow + e * 4) = word;
        if (e == 0)
          *reinterpret_cast<uint32_t*>(block + (is_v ? KvBlock<D>::kVPairs : KvBlock<D>::kPairs) + at.slot * 4) = pair;
      }
    }
    if (is_q) {
      uint4 o = make_uint4(0, 0, 0, 0);
      if (!none)
        o = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
      *reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + static_cast<int64_t>(row) * D + e * 8) = o;
    }
  }
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
  constexpr int kAtOnce = 32 / kLanes;
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int e = lane % kLanes;
  if (blockIdx.y == 0)
    for (int64_t i = t * kAppendThreads + threadIdx.x; i < c.num_reqs; i += int64_t(gridDim.x) * kAppendThreads)
      check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
  const Place at = place_of<D>(c, t);
  if (at.r >= 0 && at.block == nullptr && lane == 0) set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
  const int rows = 2 * c.num_kv_heads;  // K heads, then V heads
#pragma unroll 2
  for (int row = (blockIdx.y * (kAppendThreads / 32) + threadIdx.x / 32) * kAtOnce + lane / kLanes; row < rows;
       row += gridDim.y * (kAppendThreads / 32) * kAtOnce) {
    const bool is_v = row >= c.num_kv_heads;
    const int h = is_v ? row - c.num_kv_heads : row;
    ple_bf16_t* out = is_v ? a.v_out : a.k_out;
    if (out == nullptr) continue;
    uint4 o = make_uint4(0, 0, 0, 0);
    if (at.block != nullptr) {
      const uint8_t* block = at.block + h * at.head_stride;
      const uint32_t word = *reinterpret_cast<const uint32_t*>(
          block + (is_v ? KvBlock<D>::kV : 0) + at.slot * KvBlock<D>::kRow + e * 4);
      const uint32_t pair = *reinterpret_cast<const uint32_t*>(
          block + (is_v ? KvBlock<D>::kVPairs : KvBlock<D>::kPairs) + at.slot * 4);
      const float scale = bf_lo(pair), offset = bf_hi(pair);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = fmaf(static_cast<float>((word >> (4 * i)) & 15u), scale, offset);
      o = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    }
    *reinterpret_cast<uint4*>(out + (t * c.num_kv_heads + h) * D + e * 8) = o;
  }
}

// A token's rows are split over as many CTAs as it takes to give every SM
// some warps: with tokens enough one CTA has them all.
dim3 row_grid(int64_t T, int rows, int D) {
  const int per_cta = kAppendThreads / (D / 8);  // rows of a CTA at once
  const int most = (rows + per_cta - 1) / per_cta;
  const int64_t want = (int64_t(num_sms()) * 8 + T - 1) / T;
  return dim3(static_cast<unsigned>(T), static_cast<unsigned>(want < most ? want : most));
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
