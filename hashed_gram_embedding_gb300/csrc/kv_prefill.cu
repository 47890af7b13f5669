// ple_kv_attention for requests of many query rows (prefill chunks): 256 rows
// against 128 positions at a time on the 5th-generation tensor cores.
//
// Work. A CTA takes 256 query rows of one request and kv head (rows are
// (token, head of the group), so a group's heads share every key) as two
// tiles of 128 - one, for heads of 256 - and walks the positions they see in tiles of 128. Rows of
// long requests come first, so that the last CTAs are short ones. Where these
// would not fill the GPU, several CTAs share the positions of one such piece of
// rows, and a second kernel joins their outputs, each with its rows' m and l,
// in the order of the positions.
//
// Mathematics. For each tile of positions, S = Q K^T (f16 operands, f32 in
// tensor memory), P = exp2(f S - m) rounded to f16 over S in tensor memory,
// O += P V (f16 operands, f32 in tensor memory). m need not be the largest
// score for that, only near it: weights and sums are floating point. So a
// tile's weights are taken with the m there is while its maximum is being
// found, and m is raised (and O scaled) between tiles, when a weight passed
// 2^11. Only a weight above 2^15, which f16 could not hold - a row's first,
// mostly - raises it at once. A raise leaves the largest weight at 2^4, so that
// what f16 cannot tell from nothing, 2^-25, is 2^-29 of it.
// Roundings: a key enters as f16(code * scale + offset), because a score of
// hundreds must not move by a bf16's 2^-8 of it; rows of Q are scaled to
// [1, 2) by a power of two (in the row's f), and a key row outside
// [2^-6, 512) by one of its own, which is multiplied back on a path of its
// own. Values and weights enter as f16 too (with bf16 the result's error was
// 0.0028 of it, now it is its own rounding's, 0.0017). A value row outside
// [2^-6, 512) is divided by a power of two, 2^k, and k added to its scores in
// log2 units: the weights that meet V, and m, are those of the shifted scores,
// the sum that divides them is that of the true ones. It is kept in units of
// 2^m while that loses nothing: with shifts in [-24, 32] m stays within 40 of
// the true scores' maximum, far inside float32's exponents. From the first
// tile on with a shift outside, it has a maximum of its own.
//
// Roles (20 warps): warps 0-3 and 4-7 each own a tile of rows, a row a
// thread: they read S, write P, scale O and write the result. Warps 8-11 turn
// the cache's codes into K operands (positions x D), warps 12-15 into V
// operands (transposed: D x positions), both K-major with 128-byte swizzle,
// two buffers each (heads of 256: one), the next tile's codes on their way
// meanwhile. Warp 16 issues the products: while one tile of rows is
// exponentiated the other's are multiplied. The order of a group of 8 elements in Q and K is (0, 4, 1, 5, 2,
// 6, 3, 7), as two masks of a word of codes give them.
//
// A code masked out where it stands is a subnormal number: one product makes
// c / 512 of it, one multiply-add code * scale + offset.
//
// Bound by latency: a tile's chain of S, weights, P V and the next S, about
// 4900 cycles for both tiles, of which their products are 2048 and their
// exponentials another 2048, side by side only in part: a tile's weights stand
// over its scores, so its next scores wait for P V (scores of 64 positions at a
// time, in two pieces, would find room; registers and instruction caches leave
// none for a third tile of rows). Measured, 32 heads on 8 kv heads of 128:
// 2048 tokens of a request on 16k positions 557 us = 926 TFLOP/s, a ragged
// prefill of 8192 tokens behind 2000 positions 339 us = 611 (its last CTAs run
// alone); 64 tokens on 65k positions 126 us. Heads of 256: 2 x 1024 tokens of
// 16 heads on 4k positions 310 us = 500 TFLOP/s.
//
// What is masked never meets what it must not: a position outside the cache
// enters as zeros, and a value that is not finite is left out of V and makes
// NaN of the rows that see it, instead of all rows of its tile.
#include "kv_attention.cuh"
#include "tensor_core.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace ple {
namespace {

constexpr int kTile = 128;        // rows of a tile, and positions
constexpr int kGroupThreads = 128;
constexpr int kThreads = 20 * 32;
// Registers a thread is launched with, and each role's share of the CTA's.
constexpr int kRegisters = 96, kRowRegisters = 120, kCodeRegisters = 88, kProductRegisters = 64;
static_assert(kRowRegisters >= kRegisters && kCodeRegisters <= kRegisters && kProductRegisters <= kRegisters,
              "rows ask for more than they start with, the others give back");
static_assert(2 * kRowRegisters + 2 * kCodeRegisters + kProductRegisters <= 5 * kRegisters, "more would never be had");
constexpr int kMaskRing = 4;      // tiles whose masks are kept
constexpr int kMaskWords = 20;
// In log2 of a weight: where a raise puts the largest, when it is due, when it cannot wait.
constexpr float kRaised = 4.0f, kRaise = 11.0f, kRaiseNow = 15.0f;

template <int D>
struct Prefill {
  // Two tiles of rows and two buffers of K and V; heads of 256 fill shared and
  // tensor memory with one of each.
  static constexpr int kRowTiles = D <= 128 ? 2 : 1, kBuffers = D <= 128 ? 2 : 1;
  static constexpr int kRows = kRowTiles * kTile;
  static constexpr int kQ = kTile * D * 2;       // bytes of an operand tile
  static constexpr int kAtK = kRowTiles * kQ;
  static constexpr int kAtV = kAtK + kBuffers * kQ;
  static constexpr int kAtMasks = kAtV + kBuffers * kQ;  // [ring][5][4] present; V not finite; K has a factor; any such; V is shifted
  static constexpr int kAtFactors = kAtMasks + kMaskRing * kMaskWords * 4;  // [ring][128] of K rows
  static constexpr int kAtShifts = kAtFactors + kMaskRing * kTile * 4;      // [ring][128] of V rows, in log2
  static constexpr int kAtBars = kAtShifts + kMaskRing * kTile * 4;
  static constexpr int kAtWords = kAtBars + 16 * 8;
  static_assert(2 * kTile + kRowTiles * D <= 512, "tensor memory");
  static constexpr int kSmem = kAtWords + 80 + 1024;         // and alignment
};

__device__ __forceinline__ uint32_t f16_mul(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t f16_mad(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Codes i and i + 4 of a word as f16 pair c / 512.
__device__ __forceinline__ uint32_t code_512ths(uint32_t word, int i) {
  return f16_mul(code_bits(word, i), i % 2 == 0 ? 0x78007800u /* 2^15 */ : 0x68006800u /* 2^11 */);
}

// log2 of what a value row of these (scale, offset) is divided by to lie in
// f16's range: 0 if its largest magnitude is in [2^-6, 512) or zero. Not below
// -90, so that a true weight stays below 2^128 (of rows smaller than 2^-96
// bits are lost), and of no matter for rows that are not finite.
__device__ __forceinline__ int value_shift(uint32_t pair) {
  const float s = bf_lo(pair), m = bf_hi(pair);
  const int e = static_cast<int>(__float_as_uint(fmaxf(fabsf(m), fabsf(fmaf(15.0f, s, m)))) >> 23);
  return static_cast<unsigned>(e - 121) < 15u || e == 0 ? 0 : min(max(e - 127, -90), 119);
}
// Shifts that the sum of a row's weights cannot follow in the units of m.
__device__ __forceinline__ bool far_shift(float shift) { return shift < -24.0f || shift > 32.0f; }

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A row's outputs times `keep`. Rare.
template <int D>
__device__ __forceinline__ void rescale_outputs(uint32_t at, float keep) {
#pragma unroll 1
  for (int q = 0; q < D / 32; ++q) {
    float o[32];
    uint32_t u[32];
    tmem_load(at + 32 * q, o);
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * keep);
    tmem_store32(at + 32 * q, u);
  }
}

// 32 weights of a row, already in tensor memory, times `keep` (a power of two). Rare.
__device__ __forceinline__ void rescale_weights(uint32_t at, float keep) {
  float w[16];
  uint32_t u[16];
  const uint32_t keep2 = f16_pair(keep, keep);
  tmem_load16(at, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) u[i] = f16_mul(__float_as_uint(w[i]), keep2);
  tmem_store16(at, u);
}

// Where pieces of rows are shared: what a piece became, and its parts' results.
struct Parts {
  int most;        // parts of a piece at most; 1: none is shared
  int4* pieces;    // [pieces][2] parts (0: no such piece), rows, tile, head; first token
  float4* sums;    // [pieces][most][rows] m; l, and the log2 of its unit
  float* outputs;  // [pieces][most][rows][D]
};

// Tiles of positions to a part at least: a CTA's start and end cost as much as some tiles.
constexpr int kPartTiles = 4;

// A CTA's share of the work.
struct Job {
  int r, tile, h;     // request, 256-row tile, kv head
  int t0, n, len;     // of the request
  int rows;           // in the tile
  int first, tiles;   // first position tile, and how many
  int block0, block_end;
  int parts;          // CTAs that share its rows
  bool clipped;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attention_prefill_kernel(const AttentionArgs a, const KvCache c, const Parts parts) {
  using L = Prefill<D>;
  using B = KvBlock<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t bar0 = base + L::kAtBars;
  const uint32_t q_full = bar0, o_full = bar0 + 8;
  auto k_full = [&](int b) { return bar0 + 16 + 8u * b; };
  auto k_free = [&](int b) { return bar0 + 32 + 8u * b; };
  auto v_full = [&](int b) { return bar0 + 48 + 8u * b; };
  auto v_free = [&](int b) { return bar0 + 64 + 8u * b; };
  auto s_full = [&](int t) { return bar0 + 80 + 8u * t; };
  auto p_full = [&](int t) { return bar0 + 96 + 8u * t; };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kAtWords);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + L::kAtWords + 4);
  Job* const job = reinterpret_cast<Job*>(smem + L::kAtWords + 8);
  static_assert(sizeof(Job) <= 60, "room in shared memory");
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int G = a.num_heads / c.num_kv_heads, hk = c.num_kv_heads;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);  // warps
    mbar_init(o_full, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(k_full(b), 4);
      mbar_init(k_free(b), 1);
      mbar_init(v_full(b), 4);
      mbar_init(v_free(b), 1);
      mbar_init(s_full(b), 1);
      mbar_init(p_full(b), 4);
    }
    mbar_fence_init();
    *abort_flag = 0;
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {  // this CTA's share: tiles of a request from the last one on, its heads side by side
    const int piece = blockIdx.x / parts.most, part = blockIdx.x - piece * parts.most;
    int left = piece, r0 = 0;
    Job x;
    x.r = -1;
    while (r0 < c.num_reqs) {
      const int r = r0 + lane;
      int64_t t0 = 0, end = 0;
      if (r < c.num_reqs) request_span(c.qsl, c.num_reqs + 1, a.T, r, &t0, &end);
      const int rows = static_cast<int>(end - t0) * G;
      const int tiles = rows >= a.many_rows ? (rows + L::kRows - 1) / L::kRows : 0;
      int sum = tiles * hk;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const unsigned past = __ballot_sync(0xffffffffu, sum > left);
      if (past != 0) {
        if (lane == __ffs(past) - 1) {
          const int at = left - (sum - tiles * hk);
          x.r = r;
          x.tile = tiles - 1 - at / hk;
          x.h = at % hk;
          x.t0 = static_cast<int>(t0);
          x.n = static_cast<int>(end - t0);
          x.len = max(__ldg(c.kv_lens + r), 0);
          x.rows = min(L::kRows, rows - x.tile * L::kRows);
          // the positions that its rows see
          const int tok0 = x.tile * L::kRows / G, tok1 = (x.tile * L::kRows + x.rows - 1) / G;
          const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_size;
          int64_t hi = a.causal ? int64_t(x.len) - x.n + tok1 + 1 : x.len;
          x.clipped = hi > room;
          hi = min(hi, room);
          int64_t lo = a.window > 0 ? int64_t(x.len) - x.n + tok0 - a.window + 1 : 0;
          lo = max(lo, int64_t(0));
          x.first = static_cast<int>(lo / kTile);
          x.tiles = hi > lo ? static_cast<int>((hi + kTile - 1) / kTile) - x.first : 0;
          x.block0 = static_cast<int>(lo / kBlockTokens);
          x.block_end = hi > 0 ? static_cast<int>((hi + kBlockTokens - 1) / kBlockTokens) : 0;
          x.parts = max(1, min(parts.most, x.tiles / kPartTiles));
          if (parts.most > 1 && part == 0) {
            parts.pieces[2 * piece] = make_int4(x.parts, x.rows, x.tile, x.h);
            parts.pieces[2 * piece + 1] = make_int4(x.t0, 0, 0, 0);
          }
          const int lo_tile = static_cast<int>(int64_t(x.tiles) * part / x.parts);
          x.tiles = static_cast<int>(int64_t(x.tiles) * (part + 1) / x.parts) - lo_tile;
          x.first += lo_tile;
          if (part >= x.parts) x.r = -1;
          *job = x;
        }
        break;
      }
      left -= __shfl_sync(0xffffffffu, sum, 31);
      r0 += 32;
    }
    if (r0 >= c.num_reqs && lane == 0) {
      job->r = -1;
      if (parts.most > 1 && part == 0) parts.pieces[2 * piece] = make_int4(0, 0, 0, 0);
    }
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const Job x = *job;
  const bool two = x.rows > kTile;  // both tiles have rows
  const int n = x.r >= 0 ? x.tiles : 0;
  auto gave_up = [&](bool ok) {
    if (!ok) {
      *abort_flag = 1;
      set_dev_err(a.dev_err, PLE_DEVERR_TIMEOUT);
    }
    return !ok;
  };
  uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + L::kAtMasks);

  if (x.r >= 0 && warp < 8) {
    // ---------------- a row a thread ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegisters));
    const int t = warp / 4;                       // tile of rows
    const int row = threadIdx.x % kGroupThreads;
    const int in_tile = t * kTile + row;
    const int flat = x.tile * L::kRows + in_tile;
    const bool live = in_tile < x.rows;
    const int token = flat / G;
    const int64_t head = static_cast<int64_t>(x.h * G + (flat - token * G)) * D;
    float factor = a.scale_log2;                  // takes a row's scores to log2 units
    if (t == 0 || two) {
      const ple_bf16_t* src = a.q + static_cast<int64_t>(x.t0 + token) * a.q_stride + head;
      uint8_t* dst = smem + t * L::kQ;
      float top = 0.0f;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = *reinterpret_cast<const uint4*>(src + 8 * i);
        float e[8];
        unpack8(v, e);
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(e[k]));
      }
      // 2^k <= top < 2^(k + 1)
      const int k = top > 0.0f && top < INFINITY ? max(ilogbf(top), -126) : 0;
      const float down = ldexpf(1.0f, -k);
      factor = ldexpf(a.scale_log2, k);
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = *reinterpret_cast<const uint4*>(src + 8 * i);
        float e[8];
        unpack8(v, e);
#pragma unroll
        for (int h = 0; h < 8; ++h) e[h] *= down;
        *reinterpret_cast<uint4*>(dst + chunk_at(kTile, row, i)) =
            make_uint4(f16_pair(e[0], e[4]), f16_pair(e[1], e[5]), f16_pair(e[2], e[6]), f16_pair(e[3], e[7]));
      }
    }
    fence_operands();
    warp_arrive(q_full);
    const int last = !live ? -1 : a.causal ? x.len - x.n + token : x.len - 1;
    const int from = a.window > 0 && last - a.window + 1 > 0 ? last - a.window + 1 : 0;
    // what every live row of the warp sees
    const int all_to = __reduce_min_sync(0xffffffffu, live ? last : INT32_MAX);
    const int all_from = __reduce_max_sync(0xffffffffu, live ? from : 0);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * kTile;
    const uint32_t o_at = tmem + lanes + 2 * kTile + t * D;
    float m = -FLT_MAX, l = 0.0f, top = -FLT_MAX;
    float lm = 0.0f;                              // once the sum has a unit of its own: l is in units of 2^lm
    bool ok = true;
    if (t == 0 || two) {
      int j = 0;
      // Tiles from j on; without `apart` up to the first that needs it, which
      // keeps what is rare out of the loop that is not.
      auto walk = [&](auto apart) {
        constexpr bool kApart = decltype(apart)::value;
#pragma unroll 1
        for (; j < n; ++j) {
          ok = wait_for(s_full(t), j & 1, abort_flag);
          if (gave_up(__all_sync(0xffffffffu, ok))) { ok = false; break; }
          fence_after();
          const int p0 = (x.first + j) * kTile;
          const uint32_t* mask = masks + (j % kMaskRing) * kMaskWords;
          const uint4 any = *reinterpret_cast<const uint4*>(mask + 12);
          const bool special = p0 < all_from || p0 + kTile - 1 > all_to || (any.x | any.y | any.z | any.w) != 0;
          if (__any_sync(0xffffffffu, top > m + kRaise)) {
            const float next = fmaxf(m, top - kRaised);
            const float keep = ex2(m - next);
            m = next;
            if constexpr (!kApart) l *= keep;
            // S(j) done means that the products of tile j - 1, issued before it, are done
            if (j > 0) rescale_outputs<D>(o_at, keep);
          }
          // a quarter of the row at a time, in a rolled loop: what the roles run
          // side by side has to fit the instruction caches (2048 rows of 32 heads
          // on 16k positions, when this was chosen: 540 us, two quarters to a turn
          // 553, four half as long again)
          auto quarter = [&](int q, auto shifted) {
            float v[32];
            tmem_load(s_at + 32 * q, v);
            float to_log2 = factor;
            const float* shifts = reinterpret_cast<const float*>(smem + L::kAtShifts) + (j % kMaskRing) * kTile + 32 * q;
            if (shifted.value || special) {
              const float* factors = reinterpret_cast<const float*>(smem + L::kAtFactors) + (j % kMaskRing) * kTile + 32 * q;
              // bits of the columns that the row may see
              const int hi = last - p0 - 32 * q, lo = from - p0 - 32 * q;  // lo..hi
              uint32_t see = hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1u;
              if (lo > 0) see &= lo >= 32 ? 0u : 0xffffffffu << lo;
              see &= mask[q];
              if ((see & mask[4 + q]) != 0) l = NAN;
              if (mask[8 + q] != 0) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= factors[i];
              }
              if constexpr (shifted.value) {
                to_log2 = 1.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], factor, shifts[i]);
              }
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((see >> i) & 1u)) v[i] = -INFINITY;
            }
            float tops[2] = {v[0], v[1]};
#pragma unroll
            for (int i = 2; i < 32; i += 2) {
              tops[0] = fmaxf(tops[0], v[i]);
              tops[1] = fmaxf(tops[1], v[i + 1]);
            }
            top = fmaxf(top, to_log2 * fmaxf(tops[0], tops[1]));
            if (__any_sync(0xffffffffu, top > m + kRaiseNow)) {  // by a power of two: weights are scaled exactly
              const float next = !(top > m + kRaised) ? m : m == -FLT_MAX ? ceilf(top) - kRaised : m + ceilf(top - m) - kRaised;
              const float keep = ex2(m - next);
              m = next;
              if constexpr (!kApart) l *= keep;
              tmem_stored();
#pragma unroll 1
              for (int k = 0; k < q; ++k) rescale_weights(s_at + 16 * k, keep);
              if (j > 0) rescale_outputs<D>(o_at, keep);
            }
            const uint64_t f2v = f2(to_log2, to_log2), m2 = f2(-m, -m);
            if constexpr (shifted.value) {  // the true weights' sum
              if constexpr (kApart) {
                float most = lm;
#pragma unroll
                for (int i = 0; i < 32; ++i) most = fmaxf(most, v[i] - shifts[i]);
                l *= ex2(lm - most);
                lm = most;
              }
              const float unit = kApart ? lm : m;
#pragma unroll
              for (int i = 0; i < 32; ++i) l += ex2(v[i] - shifts[i] - unit);
            }
            uint64_t sum = f2(0.0f, 0.0f);
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float e0, e1;
              f2_split(f2_fma(f2(v[i], v[i + 1]), f2v, m2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum = f2_add(sum, f2(e0, e1));
              p[i >> 1] = f16_pair(e0, e1);
            }
            tmem_store16(s_at + 16 * q, p);  // over columns already read
            float l0, l1;
            f2_split(sum, l0, l1);
            if constexpr (!shifted.value) l += l0 + l1;
          };
          if (kApart || (special && (mask[16] | mask[17] | mask[18] | mask[19]) != 0)) {
            if constexpr (!kApart) {
              // looked at here, where it is rare: four more words of masks cost 5 %
              const float4 sh = reinterpret_cast<const float4*>(smem + L::kAtShifts)[(j % kMaskRing) * (kTile / 4) + lane];
              if (__any_sync(0xffffffffu, far_shift(sh.x) || far_shift(sh.y) || far_shift(sh.z) || far_shift(sh.w))) return;
            }
#pragma unroll 1
            for (int q = 0; q < 4; ++q) quarter(q, std::true_type{});
          } else if constexpr (!kApart) {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) quarter(q, std::false_type{});
          }
          tmem_stored();
          fence_before();
          warp_arrive(p_full(t));
        }
      };
      walk(std::false_type{});
      lm = m;
      if (ok && j < n) walk(std::true_type{});
      if (n > 0 && ok) {
        ok = wait_for(o_full, 0, abort_flag);
        ok = !gave_up(__all_sync(0xffffffffu, ok));
        fence_after();
      }
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * L::kRows + in_tile;
      if (x.parts > 1) parts.sums[slot] = make_float4(m, l, lm, 0.0f);
      const float inv = l == 0.0f ? 0.0f : 1.0f / l * ex2(m - lm);
      ple_bf16_t* dst = a.out + static_cast<int64_t>(x.t0 + token) * a.out_stride + head;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        if (n > 0 && ok) tmem_load(o_at + 32 * q, o);
        else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.0f;
        }
        if (x.parts > 1) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(parts.outputs + slot * D + 32 * q + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        } else if (live) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(dst + 32 * q + i) =
                make_uint4(pack2(o[i] * inv, o[i + 1] * inv), pack2(o[i + 2] * inv, o[i + 3] * inv),
                           pack2(o[i + 4] * inv, o[i + 5] * inv), pack2(o[i + 6] * inv, o[i + 7] * inv));
        }
      }
    }
  } else if (x.r >= 0 && warp < 16) {
    // ---------------- codes to operands ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCodeRegisters));
    const int id = threadIdx.x % kGroupThreads, dw = warp & 3;
    const int per_page = c.page_size / kBlockTokens;
    const int32_t* table = c.block_table + static_cast<int64_t>(x.r) * c.max_pages;
    const uint8_t* const cache = c.base;
    auto block_at = [&](int b) {
      if (b < x.block0 || b >= x.block_end) return -1;
      const int col = b / per_page;
      const int64_t page = __ldg(table + col);
      if (page < 0 || page >= c.num_pages) {
        set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
        return -1;
      }
      return static_cast<int>((page * hk + x.h) * per_page + (b - col * per_page));
    };
    constexpr int kWords = D / 8;  // words of a row
    bool ok = true;
    if (warp < 12) {
      // K: a position a thread
      if (x.clipped && id == 0) set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
      const int slot = id % kBlockTokens;
      int block;                    // of the tile to fetch
      uint4 next[kWords / 4];
      uint32_t next_kp, next_vp;
      bool next_here;
      auto find = [&](int j) { block = j < n ? block_at((x.first + j) * (kTile / kBlockTokens) + id / kBlockTokens) : -1; };
      auto fetch = [&](int j) {
        next_kp = next_vp = 0;
        next_here = block >= 0 && (x.first + j) * kTile + id < x.len;
        if (next_here) {
          const uint8_t* p = cache + static_cast<int64_t>(block) * B::kBytes;
#pragma unroll
          for (int i = 0; i < kWords / 4; ++i) next[i] = __ldg(reinterpret_cast<const uint4*>(p + slot * B::kRow) + i);
          next_kp = __ldg(reinterpret_cast<const uint32_t*>(p + B::kPairs + slot * 4));
          next_vp = __ldg(reinterpret_cast<const uint32_t*>(p + B::kVPairs + slot * 4));
        }
      };
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) next[i] = make_uint4(0, 0, 0, 0);
      find(0);
      fetch(0);
      find(1);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int b = j % L::kBuffers;
        uint4 codes[kWords / 4];
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) codes[i] = next[i];
        const uint32_t kp = next_kp, vp = next_vp;
        const bool here = next_here;
        fetch(j + 1);  // on its way while this tile is laid out
        find(j + 2);
        // the key row's largest magnitude decides whether it needs a factor
        float ks = bf_lo(kp), km = bf_hi(kp);
        const float most = fmaxf(fabsf(km), fabsf(fmaf(15.0f, ks, km)));
        const bool odd = most > 0.0f && most < INFINITY && !(most >= 0.015625f && most < 512.0f);
        const bool finite = (vp & 0x7F80u) != 0x7F80u && (vp & 0x7F800000u) != 0x7F800000u;
        const uint32_t present = __ballot_sync(0xffffffffu, here);
        const uint32_t broken = __ballot_sync(0xffffffffu, !finite);
        const uint32_t scaled = __ballot_sync(0xffffffffu, odd);
        const int shift = value_shift(vp);
        const uint32_t shifted = __ballot_sync(0xffffffffu, shift != 0);
        ok = wait_for(k_free(b), ((j / L::kBuffers) & 1) ^ 1u, abort_flag);
        if (gave_up(__all_sync(0xffffffffu, ok))) break;
        float* factors = reinterpret_cast<float*>(smem + L::kAtFactors) + (j % kMaskRing) * kTile;
        if (scaled != 0) {
          const int k = odd ? max(ilogbf(most), -126) : 0;
          factors[id] = ldexpf(1.0f, k);
          ks *= ldexpf(1.0f, -k);
          km *= ldexpf(1.0f, -k);
        } else {
          factors[id] = 1.0f;
        }
        reinterpret_cast<float*>(smem + L::kAtShifts)[(j % kMaskRing) * kTile + id] = static_cast<float>(shift);
        if (lane == 0) {
          uint32_t* mask = masks + (j % kMaskRing) * kMaskWords + dw;
          mask[0] = present;
          mask[4] = broken;
          mask[8] = scaled;
          mask[12] = ~present | broken | scaled | shifted;
          mask[16] = shifted;
        }
        const uint32_t s512 = f16_pair(512.0f * ks, 512.0f * ks), off = f16_pair(km, km);
        uint8_t* dst = smem + L::kAtK + b * L::kQ;
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 v;
            v.x = f16_mad(code_512ths(w[k], 0), s512, off);
            v.y = f16_mad(code_512ths(w[k], 1), s512, off);
            v.z = f16_mad(code_512ths(w[k], 2), s512, off);
            v.w = f16_mad(code_512ths(w[k], 3), s512, off);
            *reinterpret_cast<uint4*>(dst + chunk_at(kTile, id, 4 * i + k)) = v;
          }
        }
        fence_operands();
        warp_arrive(k_full(b));
      }
    } else {
      // V: eight positions and D / 64 words of them a thread; neighbouring
      // lanes hold neighbouring eights, whose chunks share a row
      constexpr int kPer = D / 64;
      const int eights = (lane & 7) + 8 * (dw >> 1);
      const int word = ((lane >> 3) + 4 * (dw & 1)) * kPer;
      int block;
      uint32_t next[8][kPer];
      uint2 next_pairs;  // of two of the eight positions, this lane's to prepare
      auto find = [&](int j) { block = j < n ? block_at((x.first + j) * (kTile / kBlockTokens) + eights / 2) : -1; };
      auto fetch = [&](int j) {
        next_pairs = make_uint2(0, 0);
        const int left = x.len - ((x.first + j) * kTile + eights * 8);  // positions of these in the cache
        if (block >= 0 && left > 0) {
          const uint8_t* p = cache + static_cast<int64_t>(block) * B::kBytes;
          const int slot = (eights & 1) * 8;
          next_pairs = __ldg(reinterpret_cast<const uint2*>(p + B::kVPairs + slot * 4) + (lane >> 3));
          // what lies behind the last position enters as zeros
          if (left <= (lane >> 3) * 2) next_pairs.x = 0;
          if (left <= (lane >> 3) * 2 + 1) next_pairs.y = 0;
          p += B::kV + slot * B::kRow + word * 4;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if constexpr (kPer == 4) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + i * B::kRow));
              next[i][0] = v.x;
              next[i][1] = v.y;
              next[i][2] = v.z;
              next[i][3] = v.w;
            } else if constexpr (kPer == 2) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + i * B::kRow));
              next[i][0] = v.x;
              next[i][1] = v.y;
            } else {
              next[i][0] = __ldg(reinterpret_cast<const uint32_t*>(p + i * B::kRow));
            }
          }
        }
      };
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < kPer; ++k) next[i][k] = 0;
      find(0);
      fetch(0);
      find(1);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int b = j % L::kBuffers;
        uint32_t codes[8][kPer];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int k = 0; k < kPer; ++k) codes[i][k] = next[i][k];
        // (512 scale, offset) of two positions a lane, then of all eight
        uint32_t s512[4], off[4];
        {
          uint32_t pair[2] = {next_pairs.x, next_pairs.y};
          float step[2], low[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // not finite: the rows that see it become NaN by the mask
            if ((pair[i] & 0x7F80u) == 0x7F80u || (pair[i] & 0x7F800000u) == 0x7F800000u) pair[i] = 0;
            const float down = __uint_as_float(static_cast<uint32_t>(127 - value_shift(pair[i])) << 23);
            step[i] = 512.0f * (bf_lo(pair[i]) * down);
            low[i] = bf_hi(pair[i]) * down;
          }
          const uint32_t steps = f16_pair(step[0], step[1]), lows = f16_pair(low[0], low[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s512[i] = __shfl_sync(0xffffffffu, steps, (lane & 7) + 8 * i);
            off[i] = __shfl_sync(0xffffffffu, lows, (lane & 7) + 8 * i);
          }
        }
        fetch(j + 1);
        find(j + 2);
        ok = wait_for(v_free(b), ((j / L::kBuffers) & 1) ^ 1u, abort_flag);
        if (gave_up(__all_sync(0xffffffffu, ok))) break;
        uint8_t* dst = smem + L::kAtV + b * L::kQ;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __byte_perm(codes[2 * i][k], codes[2 * i + 1][k], half == 0 ? 0x5410 : 0x7632);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 v;
              v.x = f16_mad(code_512ths(y[0], q), s512[0], off[0]);
              v.y = f16_mad(code_512ths(y[1], q), s512[1], off[1]);
              v.z = f16_mad(code_512ths(y[2], q), s512[2], off[2]);
              v.w = f16_mad(code_512ths(y[3], q), s512[3], off[3]);
              *reinterpret_cast<uint4*>(dst + chunk_at(D, (word + k) * 8 + half * 4 + q, eights)) = v;
            }
          }
        fence_operands();
        warp_arrive(v_full(b));
      }
    }
  } else if (x.r >= 0) {
    // ---------------- products ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProductRegisters));
    if (warp == 16 && n > 0) {
      const uint32_t acc = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_op = operand(base), k_op = operand(base + L::kAtK), v_op = operand(base + L::kAtV);
      constexpr uint32_t kTileOp = L::kQ >> 4;
      auto scores = [&](int t, int b) {  // S = Q K^T of one tile of rows
        if (elected()) {
          const uint32_t d = acc + t * kTile, q = q_op + t * kTileOp, k = k_op + b * kTileOp;
          mma_smem<false>(d, q, k, idesc(kTile, 0));
#pragma unroll
          for (int i = 1; i < D / 16; ++i) {
            const uint32_t at = ((i / 4) * kTile * 128 + (i % 4) * 32) >> 4;
            mma_smem<true>(d, q + at, k + at, idesc(kTile, 0));
          }
          mma_commit(s_full(t));
        }
        __syncwarp();
      };
      auto outputs = [&](int t, int b, bool add) {  // O += P V
        if (elected()) {
          const uint32_t d = acc + 2 * kTile + t * D, p = acc + t * kTile, v = v_op + b * kTileOp;
#pragma unroll
          for (int i = 0; i < kTile / 16; ++i)
            mma_tmem(d, p + 8 * i, v + (((i / 4) * D * 128 + (i % 4) * 32) >> 4), idesc(D, 0), i > 0 || add);
        }
        __syncwarp();
      };
      auto commit = [&](uint32_t bar) {
        if (elected()) mma_commit(bar);
        __syncwarp();
      };
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        const bool ok = wait_for(bar, parity, abort_flag);
        return __all_sync(0xffffffffu, ok) != 0;
      };
      bool ok = wait_all(q_full, 0) && wait_all(k_full(0), 0);
      if (ok) {
        fence_after();
        scores(0, 0);
        if (two) scores(1, 0);
        commit(k_free(0));
      }
#pragma unroll 1
      for (int j = 0; ok && j < n; ++j) {
        const int b = j % L::kBuffers, nb = (j + 1) % L::kBuffers;
        const bool more = j + 1 < n;
        ok = wait_all(v_full(b), (j / L::kBuffers) & 1) && wait_all(p_full(0), j & 1);
        if (!ok) break;
        fence_after();
        outputs(0, b, j > 0);
        if constexpr (L::kRowTiles == 1) commit(v_free(b));
        if (more) {
          ok = wait_all(k_full(nb), ((j + 1) / L::kBuffers) & 1);
          if (!ok) break;
          fence_after();
          scores(0, nb);
        }
        if (two) {
          ok = wait_all(p_full(1), j & 1);
          if (!ok) break;
          fence_after();
          outputs(1, b, j > 0);
        }
        if constexpr (L::kRowTiles == 2) commit(v_free(b));
        if (more) {
          if (two) scores(1, nb);
          commit(k_free(nb));
        }
      }
      gave_up(ok);
      // every product issued has completed once this flips
      commit(o_full);
      wait_for(o_full, 0, nullptr);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// A row a warp: the parts' outputs, weighted by how far each one's m is below
// the largest, and their sums by their own units.
constexpr int kJoinWarps = 8, kJoinRows = 32;  // rows of a CTA

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
attention_join_kernel(const AttentionArgs a, const KvCache c, const Parts parts) {
  pdl_wait();
  pdl_trigger();
  constexpr int kRows = Prefill<D>::kRows;
  const int piece = blockIdx.x / (kRows / kJoinRows), row0 = blockIdx.x % (kRows / kJoinRows) * kJoinRows;
  const int4 x = parts.pieces[2 * piece];
  const int count = x.x, rows = x.y, t0 = parts.pieces[2 * piece + 1].x;
  if (count <= 1) return;
  const int lane = threadIdx.x & 31, G = a.num_heads / c.num_kv_heads;
  constexpr int kMine = D / 32;  // columns of a lane
  for (int row = row0 + threadIdx.x / 32; row < min(row0 + kJoinRows, rows); row += kJoinWarps) {
    const int64_t slot = static_cast<int64_t>(piece) * parts.most * kRows + row;
    float4 ml = make_float4(-FLT_MAX, 0.0f, -FLT_MAX, 0.0f);
    if (lane < count) ml = parts.sums[slot + lane * kRows];
    float most = ml.x, unit = ml.z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      unit = fmaxf(unit, __shfl_xor_sync(0xffffffffu, unit, o));
    }
    const float w = ex2(ml.x - most);
    float sum = ex2(ml.z - unit) * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float acc[kMine] = {};
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const float* from = parts.outputs + (slot + i * kRows) * D + lane * kMine;
      const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
      for (int k = 0; k < kMine; k += 2) {
        const float2 v = *reinterpret_cast<const float2*>(from + k);
        acc[k] = fmaf(wi, v.x, acc[k]);
        acc[k + 1] = fmaf(wi, v.y, acc[k + 1]);
      }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum * ex2(most - unit);
    const int flat = x.z * kRows + row, token = flat / G;
    ple_bf16_t* dst = a.out + static_cast<int64_t>(t0 + token) * a.out_stride +
                      static_cast<int64_t>(x.w * G + (flat - token * G)) * D + lane * kMine;
#pragma unroll
    for (int i = 0; i < kMine; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack2(acc[i] * inv, acc[i + 1] * inv);
  }
}

template <int D>
cudaError_t launch(const AttentionArgs& a, const KvCache& c, uint8_t* room, size_t room_bytes, cudaStream_t stream) {
  constexpr int kRows = Prefill<D>::kRows;
  const auto kernel = attention_prefill_kernel<D>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Prefill<D>::kSmem);
  if (err != cudaSuccess) return err;
  // no more pieces than this: every request's last one may be short
  const int group = a.num_heads / c.num_kv_heads;
  const int64_t rows = a.T * group;
  const int64_t requests = rows / a.many_rows < c.num_reqs ? rows / a.many_rows : c.num_reqs;
  const int64_t pieces = (requests == 1 ? (rows + kRows - 1) / kRows : rows / kRows + requests) * c.num_kv_heads;
  // Parts: what makes the fullest turns of all SMs, in tiles of the longest
  // context that the table has room for; a CTA's start and end cost some 6 tiles.
  constexpr size_t kPartBytes = kRows * (D * sizeof(float) + sizeof(float4));
  const int64_t cap = static_cast<int64_t>((room_bytes - 1024) / (kPartBytes + 2 * sizeof(int4)));
  int64_t seen = static_cast<int64_t>(c.max_pages) * c.page_size;
  if (a.window > 0) seen = std::min(seen, static_cast<int64_t>(a.window) + kRows / group + 1);
  const int64_t tiles = seen / kTile + 1;
  int most = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= 32 && (n == 1 || (pieces * n <= cap && n * kPartTiles <= tiles)); ++n) {
    const int64_t turns = (pieces * n + num_sms() - 1) / num_sms(), cost = turns * ((tiles + n - 1) / n + 6);
    if (cost < least) {
      least = cost;
      most = n;
    }
  }
  Parts parts{most, nullptr, nullptr, nullptr};
  if (most > 1) {
    parts.pieces = reinterpret_cast<int4*>(room);
    parts.sums = reinterpret_cast<float4*>(room + (pieces * 2 * sizeof(int4) + 255) / 256 * 256);
    parts.outputs = reinterpret_cast<float*>(parts.sums + pieces * most * kRows);
  }
  const cudaError_t run = launch_kernel(kernel, dim3(static_cast<unsigned>(pieces * most)), dim3(kThreads),
                                        Prefill<D>::kSmem, stream, 1, a, c, parts);
  if (run != cudaSuccess || most == 1) return run;
  return launch_kernel(attention_join_kernel<D>, dim3(static_cast<unsigned>(pieces * (kRows / kJoinRows))),
                       dim3(kJoinWarps * 32), 0, stream, 1, a, c, parts);
}

}  // namespace

cudaError_t launch_prefill(const AttentionArgs& a, const KvCache& c, int head_dim, void* room, size_t room_bytes,
                           cudaStream_t stream) {
  uint8_t* at = static_cast<uint8_t*>(room);
  return head_dim == 64    ? launch<64>(a, c, at, room_bytes, stream)
         : head_dim == 128 ? launch<128>(a, c, at, room_bytes, stream)
                           : launch<256>(a, c, at, room_bytes, stream);
}

}  // namespace ple
