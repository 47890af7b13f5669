// The paged 4-bit key/value cache: block layout, the arguments that find a
// token's place in it, and their checks (ple_kv_append, ple_kv_read,
// ple_kv_attention).
#pragma once

#include "common.cuh"

namespace ple {

constexpr int kBlockTokens = 16;

// Byte offsets inside a block of 16 tokens of one head.
template <int D>
struct KvBlock {
  static constexpr int kRow = D / 2;                    // codes of one token
  static constexpr int kV = kBlockTokens * kRow;        // V codes
  static constexpr int kPairs = 2 * kV;                 // K, then V (scale, offset) pairs
  static constexpr int kVPairs = kPairs + kBlockTokens * 4;
  static constexpr int kBytes = kPairs + 2 * kBlockTokens * 4;
};

struct KvCache {
  uint8_t* base;
  int64_t num_pages;
  int page_size;
  int num_kv_heads;
  const int32_t* block_table;
  int max_pages;
  const int32_t* qsl;
  int num_reqs;
  const int32_t* kv_lens;
};

// Block of position p of request r and head h, or nullptr for a position
// the table does not place in the cache.
template <int D>
__device__ __forceinline__ uint8_t* kv_block(const KvCache& c, int r, int64_t p, int h) {
  if (p < 0) return nullptr;
  const int64_t col = p / c.page_size;
  if (col >= c.max_pages) return nullptr;
  const int64_t page = __ldg(c.block_table + static_cast<int64_t>(r) * c.max_pages + col);
  if (page < 0 || page >= c.num_pages) return nullptr;
  const int per_head = c.page_size / kBlockTokens;
  const int64_t block = (page * c.num_kv_heads + h) * per_head + (p - col * c.page_size) / kBlockTokens;
  return c.base + block * KvBlock<D>::kBytes;
}

// Request of token t, found by a whole warp (32-way search of qsl, two
// rounds of loads for up to 1023 requests): the last r with qsl[r] <= t, or
// -1 for padding tokens (t < qsl[0] or t >= qsl[num_reqs]).
__device__ __forceinline__ int request_of(const int32_t* __restrict__ qsl, int num_reqs, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = num_reqs + 1;  // the count of entries <= t lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int p = lo + lane * step;
    const bool le = p < hi && static_cast<int64_t>(__ldg(qsl + p)) <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    if (k == 0) break;
    const int next = lo + (k - 1) * step + 1;
    hi = min(lo + k * step, hi);
    lo = next;
  }
  return lo == 0 || lo > num_reqs ? -1 : lo - 1;
}

// Host checks shared by the cache's entry points.
inline ple_status check_cache(const char* name, const void* cache, int64_t num_pages, int page_size,
                              const int32_t* block_table, int max_pages, const int32_t* qsl,
                              int num_reqs, const int32_t* kv_lens, int num_kv_heads, int head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(PLE_ERR_UNSUPPORTED, "%s: head_dim %d (64, 128 or 256)", name, head_dim);
  if (page_size <= 0 || page_size % kBlockTokens != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: page_size %d is not a multiple of 16", name, page_size);
  if (num_pages < 0 || max_pages < 0 || num_reqs < 1 || num_kv_heads < 1)
    return fail(PLE_ERR_INVALID_ARG, "%s: num_pages %lld, max_pages %d, num_reqs %d, num_kv_heads %d",
                name, static_cast<long long>(num_pages), max_pages, num_reqs, num_kv_heads);
  if (qsl == nullptr || kv_lens == nullptr || (block_table == nullptr && max_pages > 0) ||
      (cache == nullptr && num_pages > 0))
    return fail(PLE_ERR_INVALID_ARG, "%s: null cache, block_table, query_start_loc or kv_lens", name);
  if (!aligned16(cache)) return fail(PLE_ERR_INVALID_ARG, "%s: cache is not 16-byte aligned", name);
  return PLE_OK;
}

}  // namespace ple
