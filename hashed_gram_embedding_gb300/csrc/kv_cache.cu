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
// fill the card, one or two when there are few and latency counts. Bound by
// memory for large steps and by latency for small ones, as long as a row
// costs few instructions: with a warp for each two rows of a token and a
// division for each element a prefill of 8600 tokens (32 + 2 x 8 heads of
// 128) took 93 us to append and read back, bound by issue. Now 72 us = 3.5
// TB/s; the append issues in 56 % of the slots and otherwise waits for memory.
// 256 x 4 tokens take 14 us, one token 5.
#include "kv_cache.cuh"

namespace ple {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kWarpsPerSm = 32;

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

// Eight float32 values, as pairs.
struct Row8 {
  uint64_t v[4];
};

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ Row8 unpack_row(uint4 v) {
  return {{f2(bf_lo(v.x), bf_hi(v.x)), f2(bf_lo(v.y), bf_hi(v.y)), f2(bf_lo(v.z), bf_hi(v.z)), f2(bf_lo(v.w), bf_hi(v.w))}};
}

__device__ __forceinline__ uint4 pack_row(const Row8& x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_split(x.v[i], lo, hi);
    w[i] = pack2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Each product and the sum rounded by itself, so that a code does not depend
// on how a compiler contracts them (pairs of products and sums it does).
__device__ __forceinline__ float sum_of_products(float a, float b, float c, float d) {
  return __fadd_rn(__fmul_rn(a, b), __fmul_rn(c, d));
}

// clamp(rint((x - offset) / scale), 0, 15) of eight values, packed. The
// quotient is taken as a product with the reciprocal, within 2^-22 of it
// relative, and rounded by adding 1.5 * 2^23; where it comes near a half, the
// division decides.
__device__ __forceinline__ uint32_t codes_of(const Row8& x, float scale, float offset) {
  constexpr float kRound = 12582912.0f;
  constexpr uint32_t kRoundBits = 0x4B400000u * 0x11111111u;  // of eight, a nibble apart
  const float inv = __frcp_rn(scale);
  const uint64_t off = f2(-offset, -offset), by = f2(inv, inv), up = f2(kRound, kRound), down = f2(-kRound, -kRound);
  uint32_t word = 0u - kRoundBits;
  float far = 0.0f;  // from the code, at most
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float q0, q1, c0, c1, d0, d1;
    f2_split(f2_mul(f2_add(x.v[i], off), by), q0, q1);
    q0 = fminf(fmaxf(q0, 0.0f), 15.0f);
    q1 = fminf(fmaxf(q1, 0.0f), 15.0f);
    const uint64_t c = f2_add(f2(q0, q1), up);
    f2_split(c, c0, c1);
    f2_split(f2_add(c, down), d0, d1);
    far = fmaxf(far, fmaxf(fabsf(q0 - d0), fabsf(q1 - d1)));
    word += __float_as_uint(c0) << (8 * i);
    word += __float_as_uint(c1) << (8 * i + 4);
  }
  if (far > 0.4999f || !(scale >= 1e-37f && scale <= 1e37f)) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[2];
      f2_split(f2_add(x.v[i], off), y[0], y[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        word |= static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(y[k], scale)), 0.0f), 15.0f)) << (8 * i + 4 * k);
    }
  }
  return word;
}

// Warp `part` of `parts` of a token takes units part, part + parts, ... of its
// rows (a unit is as many rows as fit a warp): queries, then keys, then values.
template <int D>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const AppendArgs a, const KvCache c, int parts) {
  using B = KvBlock<D>;
  constexpr int kLanes = D / 8;          // lanes of a row
  constexpr int kAtOnce = 32 / kLanes;   // rows of a unit
  pdl_wait();
  pdl_trigger();
  const int64_t id = (int64_t(blockIdx.x) * kAppendThreads + threadIdx.x) / 32;
  const int64_t t = id / parts;
  if (t >= a.T) return;
  int unit = static_cast<int>(id - t * parts);
  const int lane = threadIdx.x & 31;
  const int e = lane % kLanes, sub = lane / kLanes;
  const int q_units = (a.num_heads + kAtOnce - 1) / kAtOnce, kv_units = (c.num_kv_heads + kAtOnce - 1) / kAtOnce;
  auto load = [&](const ple_bf16_t* rows, int h, int heads) {
    return h < heads ? *reinterpret_cast<const uint4*>(rows + h * D + e * 8) : make_uint4(0, 0, 0, 0);
  };
  const ple_bf16_t* q = a.q + t * a.q_stride;
  const ple_bf16_t* k = a.k + t * a.k_stride;
  const ple_bf16_t* v = a.v + t * a.v_stride;
  // the first rows are on their way while the token is looked up
  uint4 raw = unit < q_units ? load(q, unit * kAtOnce + sub, a.num_heads) : make_uint4(0, 0, 0, 0);
  if (unit == 0)
    for (int64_t i = t * 32 + lane; i < c.num_reqs; i += a.T * 32) check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
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
  // factors of a lane's elements: of themselves, and of their partners
  // (the sign in it); interleaved, cosines and sines of four pairs
  Row8 co, si;
#pragma unroll
  for (int i = 0; i < 4; ++i) { co.v[i] = f2(1.0f, 1.0f); si.v[i] = f2(0.0f, 0.0f); }
  if (turns) {
    const float* cs = a.cos_sin + angle * a.rot + (a.interleaved ? e * 4 : (first ? e : e - apart) * 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i == 1 && a.interleaved) break;
      const float4 x = __ldg(reinterpret_cast<const float4*>(cs) + i);
      const float4 y = __ldg(reinterpret_cast<const float4*>(cs + half) + i);
      const float sign = !a.interleaved && first ? -1.0f : 1.0f;
      co.v[2 * i] = f2(x.x, x.y);
      co.v[2 * i + 1] = f2(x.z, x.w);
      si.v[2 * i] = f2(sign * y.x, sign * y.y);
      si.v[2 * i + 1] = f2(sign * y.z, sign * y.w);
    }
  }
  const int partner = lane - e + (!turns ? e : first ? e + apart : e - apart);
  // All lanes of the warp call.
  auto rotated = [&](uint4 raw) {
    Row8 x = unpack_row(raw);
    if (a.cos_sin == nullptr) return x;
    if (a.interleaved) {
      if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u, w, cc[2], ss[2];
          f2_split(x.v[i], u, w);
          f2_split(co.v[i / 2], cc[0], cc[1]);
          f2_split(si.v[i / 2], ss[0], ss[1]);
          const float cv = cc[i % 2], sv = ss[i % 2];
          x.v[i] = f2(sum_of_products(u, cv, w, -sv), sum_of_products(w, cv, u, sv));
        }
      }
      return x;
    }
    uint4 other;
    other.x = __shfl_sync(0xffffffffu, raw.x, partner);
    other.y = __shfl_sync(0xffffffffu, raw.y, partner);
    other.z = __shfl_sync(0xffffffffu, raw.z, partner);
    other.w = __shfl_sync(0xffffffffu, raw.w, partner);
    if (turns) {
      const Row8 y = unpack_row(other);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x0, x1, y0, y1, c0, c1, s0, s1;
        f2_split(x.v[i], x0, x1);
        f2_split(y.v[i], y0, y1);
        f2_split(co.v[i], c0, c1);
        f2_split(si.v[i], s0, s1);
        x.v[i] = f2(sum_of_products(x0, c0, y0, s0), sum_of_products(x1, c1, y1, s1));
      }
    }
    return x;
  };
  auto store = [&](const Row8& x, int h, int codes, int pairs) {  // quantised, at the token's place
    float lo, hi, y0, y1;
    f2_split(x.v[0], y0, y1);
    lo = min_nan(y0, y1);
    hi = max_nan(y0, y1);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      f2_split(x.v[i], y0, y1);
      lo = min_nan(lo, min_nan(y0, y1));
      hi = max_nan(hi, max_nan(y0, y1));
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (h >= c.num_kv_heads || none || at.block == nullptr) return;
    uint8_t* block = at.block + h * at.head_stride;
    const uint32_t pair = pack2(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f), lo);  // (scale, offset)
    const float scale = bf_lo(pair);
    const uint32_t word = scale > 0.0f ? codes_of(x, scale, bf_hi(pair)) : 0u;
    *reinterpret_cast<uint32_t*>(block + codes + at.slot * B::kRow + e * 4) = word;
    if (e == 0) *reinterpret_cast<uint32_t*>(block + pairs + at.slot * 4) = pair;
  };
  for (; unit < q_units; unit += parts) {
    const int h = unit * kAtOnce + sub;
    const uint4 next = unit + parts < q_units ? load(q, h + parts * kAtOnce, a.num_heads) : make_uint4(0, 0, 0, 0);
    const Row8 x = rotated(raw);
    raw = next;
    if (h < a.num_heads)
      *reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + h * D + e * 8) = none ? make_uint4(0, 0, 0, 0) : pack_row(x);
  }
#pragma unroll 2
  for (unit -= q_units; unit < kv_units; unit += parts) {
    const int h = unit * kAtOnce + sub;
    store(rotated(load(k, h, c.num_kv_heads)), h, 0, B::kPairs);
  }
#pragma unroll 2
  for (unit -= kv_units; unit < kv_units; unit += parts) {
    const int h = unit * kAtOnce + sub;
    store(unpack_row(load(v, h, c.num_kv_heads)), h, B::kV, B::kVPairs);
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
kv_read_kernel(const ReadArgs a, const KvCache c, int parts) {
  using B = KvBlock<D>;
  constexpr int kLanes = D / 8;
  constexpr int kAtOnce = 32 / kLanes;
  pdl_wait();
  pdl_trigger();
  const int64_t id = (int64_t(blockIdx.x) * kAppendThreads + threadIdx.x) / 32;
  const int64_t t = id / parts;
  if (t >= a.T) return;
  const int part = static_cast<int>(id - t * parts);
  const int lane = threadIdx.x & 31;
  const int e = lane % kLanes;
  if (part == 0)
    for (int64_t i = t * 32 + lane; i < c.num_reqs; i += a.T * 32) check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
  const Place at = place_of<D>(c, t);
  if (at.r >= 0 && at.block == nullptr && lane == 0) set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
#pragma unroll 4
  for (int h = part * kAtOnce + lane / kLanes; h < c.num_kv_heads; h += parts * kAtOnce) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      ple_bf16_t* out = kv == 0 ? a.k_out : a.v_out;
      if (out == nullptr) continue;
      uint4 o = make_uint4(0, 0, 0, 0);
      if (at.block != nullptr) {
        const uint8_t* block = at.block + h * at.head_stride;
        const uint32_t word = *reinterpret_cast<const uint32_t*>(block + kv * B::kV + at.slot * B::kRow + e * 4);
        const uint32_t pair = *reinterpret_cast<const uint32_t*>(block + (kv == 0 ? B::kPairs : B::kVPairs) + at.slot * 4);
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
}

// Warps a token's units are split over: one, unless the tokens are too few to
// give every SM its share of warps.
int parts_of(int64_t T, int units) {
  const int64_t want = (int64_t(num_sms()) * kWarpsPerSm + T - 1) / T;
  return static_cast<int>(want < units ? want : units);
}

dim3 warp_grid(int64_t T, int parts) {
  return dim3(static_cast<unsigned>((T * parts * 32 + kAppendThreads - 1) / kAppendThreads));
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
  if (q != nullptr) {
    const int64_t wide = int64_t(num_heads) * head_dim * 2, narrow = int64_t(num_kv_heads) * head_dim * 2;
    const RowSpan to{q_out, num_tokens, q_out_stride * 2, wide};
    if ((!(q == q_out && q_stride == q_out_stride) && rows_overlap(to, {q, num_tokens, q_stride * 2, wide})) ||
        rows_overlap(to, {k, num_tokens, k_stride * 2, narrow}) || rows_overlap(to, {v, num_tokens, v_stride * 2, narrow}))
      return fail(PLE_ERR_INVALID_ARG, "%s: q_out overlaps k, v, or q without being it", name);
  }
  if (cos_sin != nullptr && num_positions < 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: num_positions %lld", name, static_cast<long long>(num_positions));
  const AppendArgs a{q, k, v, q_out, q_stride, k_stride, v_stride, q_out_stride, num_tokens, num_heads,
                     cos_sin, num_positions, cos_sin != nullptr ? rotary_dim : 0, interleaved != 0,
                     positions, dev_err};
  const KvCache c{static_cast<uint8_t*>(cache), num_pages, page_size, num_kv_heads, block_table,
                  max_pages, query_start_loc, num_reqs, kv_lens};
  const int at_once = 256 / head_dim;  // rows of a warp
  const int parts = parts_of(num_tokens, (num_heads + at_once - 1) / at_once + 2 * ((num_kv_heads + at_once - 1) / at_once));
  const auto kernel = head_dim == 64 ? kv_append_kernel<64> : head_dim == 128 ? kv_append_kernel<128> : kv_append_kernel<256>;
  return check_cuda(launch_kernel(kernel, warp_grid(num_tokens, parts), dim3(kAppendThreads), 0, stream, 1, a, c, parts), name);
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
  const int parts = parts_of(num_tokens, (num_kv_heads + 256 / head_dim - 1) / (256 / head_dim));
  const auto kernel = head_dim == 64 ? kv_read_kernel<64> : head_dim == 128 ? kv_read_kernel<128> : kv_read_kernel<256>;
  return check_cuda(launch_kernel(kernel, warp_grid(num_tokens, parts), dim3(kAppendThreads), 0, stream, 1, a, c, parts), name);
}
