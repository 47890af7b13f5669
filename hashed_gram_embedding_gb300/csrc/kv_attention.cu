// ple_kv_attention: grouped-query attention over the paged 4-bit cache.
#include "kv_attention.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

namespace ple {
namespace {

// ---------------------------------------------------------------------------
// Few query rows: the cache split over the card
// ---------------------------------------------------------------------------
// Work. An item is (request, tile of 8 NT query rows, kv head); its cost is
// the number of 32-token steps of the cache it reads. The steps of all items
// lie on one line, cut into equal pieces, one a warp, so a single long request
// and hundreds of ragged ones load the card alike; every warp finds its piece
// from query_start_loc and kv_lens itself (one launch, no plan on the host).
// An item that a cut falls into leaves partial results (row maxima, sums,
// unnormalised outputs, as they lie in a warp's registers) in the workspace;
// the piece that arrives last in its group of eight joins the group, the group
// that arrives last joins the groups, and so on, each in the order of the
// pieces: results do not depend on timing.
//
// Warps share nothing. Each has a ring of stages in shared memory (a stage is
// a step: two cache blocks, each one bulk copy) and fills it itself; no warp
// ever waits for another, and a warp's next item is looked up and its first
// copies fly before the last one's results are written. (A producer warp for
// seven others, which meet where an item ends, took 355 us for the first case
// below: steps handed out in turn are held up by the slowest.)
//
// Measured, 32 heads on 8 kv heads of 128: 256 ragged requests of up to 8192
// positions, a token each, 235 us = 5.7 TB/s; 4 tokens each on up to 4096
// positions 169 us = 3.7 TB/s (16 rows: twice the products for the same
// bytes); one token on 131071 positions 50 us = 2.8 TB/s (start, lookups and
// three levels of joining, which on 700 positions take 12.8 us). Bound by
// issue and by latency: on up to 2048 positions and a cold cache 56 % of the
// issue slots, 25 % of the matrix pipe and 57 % of the memory's time are in
// use with a token a request, 48, 35 and 42 % with four.
//
// Products, on warp-wide matrix instructions (16 x 8 x 16, f32 sums; reading
// the cache and unpacking it, not their rate, is the bound):
//   S^T = K Q^T     16 tokens x 8 query rows, f16
//   O^T = V^T P^T   16 elements x 8 query rows, f16
// so that a group of up to 8 query heads fills a tile, and the codes are the
// A operand of both. Unpacking a word of 8 codes:
//   Masked out where they stand, a byte's codes are subnormal numbers that no
//   bit has to be added to: bits 0-3 of a half are c 2^-24 as f16 (c 2^-133
//   as bf16), bits 4-7 sixteen times that. So a word of eight codes takes
//   four masks and one shift by a byte.
//   K: f16 subnormals multiply as they are; the query elements that meet the
//     second kind are divided by 16, and of 2^24 what the query rows leave
//     goes into the rows' factors and the keys' scales.
//   V: f16 subnormals as they are, too; the sums are multiplied by 2^24, or
//     2^20, at the end. Where a step has scales outside [2^-9, 2^10), whose
//     weights f16 would not hold or lose bits of, weights are bf16, and so are
//     codes, multiplied by 2^115 to meet them among the normal numbers.
// Query rows are scaled to [2^15, 2^16) by a power of two each, which keeps f16
// exact for bf16 queries: elements below 2^-28 of the row's largest, or 2^-24
// where they are divided by 16, lose bits. Scale and offset of a token meet
// the float32 sums instead of its elements:
//   <q, K_t> = s_t sum_d q_d c_td + m_t sum_d q_d
//   sum_t p_t V_t = sum_t p'_t c_t - 8 sum_t p'_t + sum_t p_t (m_t + 8 s_t),  p' = f16(p s)
// p' is the only rounding to fewer bits (2^-11 of it, or 2^-25; bf16: 2^-8 of
// it, with which the result's error was 0.0024 of it throughout, now it is its
// own rounding's, 0.0017). It meets codes centred on 8, so that an offset far
// from zero costs no precision; sum p' is one more row of the product, by
// constants. p is at most 2^6.
// The contraction index of a product may run in any order: a lane's 16 bytes
// of a K row are 32 neighbouring elements, and the query's fragments follow
// that order; two tokens' V bytes are interleaved with one permute a word.
// Token rows are taken in the order t ^ (t >> 1 & 1), which lets the V loads
// of neighbouring lanes fall on different banks.
constexpr int kStepTokens = 2 * kBlockTokens;

// NT tiles of 8 query rows. One CTA an SM; its warps follow from the registers
// of a warp's outputs, D NT / 4 a thread: 16 of 128 registers, 12 of 168, or 8;
// the rings take the shared memory that is left.

template <int D, int NT>
struct Split {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStage = 2 * KvBlock<D>::kBytes;
  static constexpr int kWarps = D == 256 || NT == 4 ? 8 : NT == 2 ? 12 : 16;
  static constexpr int kStages = D == 256 ? (NT == 1 ? 3 : 2) : D == 64 ? 5 : 3 + NT / 4;
  static constexpr bool kQRegs = NT == 1;            // query fragments in registers
  static constexpr int kFrags = kQRegs ? 0 : NT * (D / 16) * 32 * 8;
  static constexpr int kRowInfo = kRows * 24;        // a query row's factor, sum, last position, place in the output
  static constexpr int kAtRows = kStages * kStage + kFrags;
  static constexpr int kAtItems = kAtRows + kRowInfo;
  static constexpr int kAtBars = kAtItems + 3 * 64;
  static constexpr int kWarpBytes = (kAtBars + kStages * 8 + 127) / 128 * 128;
  static constexpr int kSmem = kWarps * kWarpBytes + 16;
  static constexpr int kSlot = kRows * (D + 2);      // floats of a partial result
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A pair of bf16 subnormals times 2^115.
__device__ __forceinline__ uint32_t times_2_115(uint32_t x) {
  return bf2_mul(x, 0x79007900u);
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// What a request asks of the kernel: steps [step0, step0 + steps) of the cache
// for each of its tiles x kv heads.
struct Span {
  int t0;          // first token
  int n;           // tokens
  int len;         // cached positions
  int step0, steps;
  int block0;      // first block that any token sees
  int tiles;
  bool clipped;    // kv_lens past the block table
};

__device__ __forceinline__ Span span_of(const AttentionArgs& a, const KvCache& c, int r, int tile_rows) {
  Span s;
  int64_t t0, end;
  request_span(c.qsl, c.num_reqs + 1, a.T, r, &t0, &end);
  s.t0 = static_cast<int>(t0);
  s.n = static_cast<int>(end - t0);
  s.len = max(__ldg(c.kv_lens + r), 0);
  const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_size;
  s.clipped = s.len > room;
  const int hi = s.clipped ? static_cast<int>(room) : s.len;
  int lo = 0;
  if (a.window > 0) {
    const int64_t first = static_cast<int64_t>(s.len) - s.n - a.window + 1;
    if (first > 0) lo = static_cast<int>(first);
  }
  s.block0 = lo / kBlockTokens;
  s.step0 = s.block0 / 2;
  s.steps = hi > lo ? (hi - 1) / kStepTokens + 1 - s.step0 : 0;
  const int rows = s.n * (a.num_heads / c.num_kv_heads);
  s.tiles = rows < a.many_rows ? (rows + tile_rows - 1) / tile_rows : 0;
  return s;
}

// An item's length on the line: what starting and joining it costs, in steps,
// then its steps; 1 for an item that only writes zeros.
constexpr int kItemCost = 6;
__device__ __forceinline__ int units_of(const Span& s) { return s.steps > 0 ? kItemCost + s.steps : 1; }

__device__ __forceinline__ int64_t weight_of(const Span& s, int hk) {
  return static_cast<int64_t>(s.tiles) * hk * units_of(s);
}

// Pieces of the line, one a warp; none so short that starting and joining it
// is most of it. One token on 700 positions, with pieces of at least 8, 4, 3, 2
// steps: 15.6, 13.5, 12.4, 14.6 us; 4 and 16 requests of as many alike.
constexpr int kMinPiece = 3;
__device__ __forceinline__ int pieces_of(int64_t W, int warps) {
  const int64_t p = (W + kMinPiece - 1) / kMinPiece;
  return p < warps ? static_cast<int>(p) : warps;
}

// A piece's share of one item.
struct Item {
  int r, tile, h, rows;
  int t0, n, len;         // of the request
  int block0, block_end;  // blocks that rows may see, up to this share's end
  int step, steps;        // first step, and how many
  int pieces, first;      // that share the item's steps, the first of them
  bool clipped;
};

// Where a warp stands on the line (in shared memory: the steps need none of it).
struct Cursor {
  int64_t W;         // the line's length
  int64_t x, x_end;  // what is left of the piece
  int64_t base;      // where request r begins
  int r;
};

constexpr int kFan = 8;  // pieces joined at a time

// Slot of an item's piece k. A piece is the first of one item that goes on,
// and a later one of one item, at most.
__device__ __forceinline__ int slot_of(int first, int k) { return 2 * (first + k) + (k == 0 ? 1 : 0); }

// An item's results in a warp's registers. Lane (g, j) holds elements
// g D / 8 + 2 u and + 1 (u < D / 16) of rows 8 n + 2 j and + 1.
template <int D, int NT>
struct Results {
  float o[NT][D / 16][4];  // (row, element): (0, 0), (1, 0), (0, 1), (1, 1)
  float m[2 * NT], l[2 * NT];
};

template <int D, int NT>
__device__ __forceinline__ void store_partial(const Results<D, NT>& x, float* slot) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int u = 0; u < D / 16; ++u)
      reinterpret_cast<float4*>(slot)[(n * (D / 16) + u) * 32 + lane] =
          make_float4(x.o[n][u][0], x.o[n][u][1], x.o[n][u][2], x.o[n][u][3]);
  if (lane < 4) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      reinterpret_cast<float4*>(slot + 8 * NT * D)[n * 4 + lane] =
          make_float4(x.m[2 * n], x.l[2 * n], x.m[2 * n + 1], x.l[2 * n + 1]);
  }
}

// Join the partial results of pieces k0, k0 + stride, ... (count of them).
template <int D, int NT>
__device__ __forceinline__ void load_joined(Results<D, NT>& x, const float* partial, int first, int k0, int stride, int count) {
  constexpr int kSlot = Split<D, NT>::kSlot;
  constexpr int kAtOnce = D / 16 < 4 ? D / 16 : 4;
  const int lane = threadIdx.x & 31, j = lane & 3;
  auto slot = [&](int k) { return partial + static_cast<int64_t>(slot_of(first, k0 + k * stride)) * kSlot; };
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float4 ml[kFan];
#pragma unroll
    for (int k = 0; k < kFan; ++k)  // past the last: it again, with no weight
      ml[k] = __ldcg(reinterpret_cast<const float4*>(slot(min(k, count - 1)) + 8 * NT * D) + n * 4 + j);
    float m0 = ml[0].x, m1 = ml[0].z;
#pragma unroll
    for (int k = 1; k < kFan; ++k) { m0 = fmaxf(m0, ml[k].x); m1 = fmaxf(m1, ml[k].z); }
    float w0[kFan], w1[kFan], l0 = 0.0f, l1 = 0.0f;
#pragma unroll
    for (int k = 0; k < kFan; ++k) {
      w0[k] = k < count ? ex2(ml[k].x - m0) : 0.0f;
      w1[k] = k < count ? ex2(ml[k].z - m1) : 0.0f;
      if (k < count) { l0 = fmaf(w0[k], ml[k].y, l0); l1 = fmaf(w1[k], ml[k].w, l1); }
    }
    x.m[2 * n] = m0; x.m[2 * n + 1] = m1;
    x.l[2 * n] = l0; x.l[2 * n + 1] = l1;
#pragma unroll
    for (int u0 = 0; u0 < D / 16; u0 += kAtOnce) {
      float4 acc[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) acc[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kFan; k += 4) {
        if (k < count) {
          float4 v[4][kAtOnce];
#pragma unroll
          for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
              v[f][u] = __ldcg(reinterpret_cast<const float4*>(slot(min(k + f, count - 1))) + (n * (D / 16) + u0 + u) * 32 + lane);
#pragma unroll
          for (int f = 0; f < 4; ++f)
            if (k + f < count)
#pragma unroll
              for (int u = 0; u < kAtOnce; ++u) {
                acc[u].x = fmaf(w0[k + f], v[f][u].x, acc[u].x); acc[u].y = fmaf(w1[k + f], v[f][u].y, acc[u].y);
                acc[u].z = fmaf(w0[k + f], v[f][u].z, acc[u].z); acc[u].w = fmaf(w1[k + f], v[f][u].w, acc[u].w);
              }
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        x.o[n][u0 + u][0] = acc[u].x; x.o[n][u0 + u][1] = acc[u].y;
        x.o[n][u0 + u][2] = acc[u].z; x.o[n][u0 + u][3] = acc[u].w;
      }
    }
  }
}

template <int D, int NT>
__device__ __forceinline__ void store_out(const Results<D, NT>& x, ple_bf16_t* out, const int64_t* row_out, int rows) {
  const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = n * 8 + 2 * j + e;
      const float l = x.l[2 * n + e], inv = l == 0.0f ? 0.0f : 1.0f / l;
      if (rr < rows) {
        uint2* dst = reinterpret_cast<uint2*>(out + row_out[rr] + g * (D / 8));
#pragma unroll
        for (int u = 0; u < D / 16; u += 2)
          dst[u / 2] = make_uint2(pack2(x.o[n][u][e] * inv, x.o[n][u][2 + e] * inv),
                                  pack2(x.o[n][u + 1][e] * inv, x.o[n][u + 1][2 + e] * inv));
      }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(Split<D, NT>::kWarps * 32, 1)
attention_split_kernel(const AttentionArgs a, const KvCache c, unsigned* __restrict__ counters,
                       float* __restrict__ partial) {
  using L = Split<D, NT>;
  using B = KvBlock<D>;
  constexpr int kRows = L::kRows, kWarps = L::kWarps;
  constexpr int kWords = D / 32;   // K words of a lane and token
  constexpr int kVWords = D / 64;  // V words of a lane and token
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int g = lane >> 2, j = lane & 3;
  uint8_t* const ring = smem + warp * L::kWarpBytes;
  uint2* const qf = reinterpret_cast<uint2*>(ring + L::kStages * L::kStage);
  float* const row_info = reinterpret_cast<float*>(ring + L::kAtRows);  // factors to log2 units, sums, ...
  int* const row_last = reinterpret_cast<int*>(row_info + 2 * kRows);
  int64_t* const row_out = reinterpret_cast<int64_t*>(row_info + 4 * kRows);
  Item* const items = reinterpret_cast<Item*>(ring + L::kAtItems);  // the present and the next
  Cursor* const cursor = reinterpret_cast<Cursor*>(items + 2);
  static_assert(sizeof(Item) <= 64 && sizeof(Item) % 8 == 0 && sizeof(Cursor) <= 64 && L::kStages <= 8, "room in shared memory and in the stages' bits");
  const uint32_t bar0 = smem_u32(ring + L::kAtBars);
  unsigned long long* const total = reinterpret_cast<unsigned long long*>(smem + kWarps * L::kWarpBytes);

  if (lane == 0) {
    for (int s = 0; s < L::kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == 0) *total = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int G = a.num_heads / c.num_kv_heads, hk = c.num_kv_heads;
  // the line's length
  int64_t W = 0;
  if (c.num_reqs <= 32) {
    if (lane < c.num_reqs) W = weight_of(span_of(a, c, lane, kRows), hk);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
  } else {
    for (int r = threadIdx.x; r < c.num_reqs; r += kWarps * 32) W += weight_of(span_of(a, c, r, kRows), hk);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
    if (lane == 0 && W > 0) atomicAdd(total, static_cast<unsigned long long>(W));
    __syncthreads();
    W = static_cast<int64_t>(*total);
  }
  const int warps = gridDim.x * kWarps;
  const int P = pieces_of(W, warps);
  const int piece = warp * gridDim.x + blockIdx.x;  // few pieces: on as many SMs
  // what is done beside the items: checks, and padding tokens' rows
  auto rest = [&]() {
    const int64_t at = int64_t(blockIdx.x) * (kWarps * 32) + threadIdx.x, all = int64_t(gridDim.x) * (kWarps * 32);
    for (int64_t i = at; i < c.num_reqs; i += all) check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
    const int64_t pad = max(__ldg(c.qsl + c.num_reqs), 0);
    const int64_t vecs = static_cast<int64_t>(a.num_heads) * (D / 8);
    for (int64_t i = pad * vecs + at; i < a.T * vecs; i += all)
      *reinterpret_cast<uint4*>(a.out + i / vecs * a.out_stride + i % vecs * 8) = make_uint4(0, 0, 0, 0);
  };
  if (piece >= P) {
    rest();
    return;
  }

  // quotients of products up to W * P, in 32 bits where they fit
  auto div = [](int64_t n, int64_t d, int64_t most) {
    return most < (int64_t(1) << 31) ? static_cast<int64_t>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d)) : n / d;
  };
  if (lane == 0) {
    Cursor at;
    at.W = W;
    at.x = div(piece * W, P, W * P);
    at.x_end = div((piece + 1) * W, P, W * P);
    at.base = 0;
    at.r = 0;
    *cursor = at;
  }
  __syncwarp();
  // The next item with steps of this piece; false if there is none.
  auto next_item = [&](Item* out) {
    const int64_t W = cursor->W, x_end = cursor->x_end;
    const int P = pieces_of(W, gridDim.x * kWarps);
    int64_t x = cursor->x, base = cursor->base;
    int r = cursor->r;
    __syncwarp();
    while (x < x_end) {
      while (r < c.num_reqs) {  // the request that x lies in
        const int64_t w = r + lane < c.num_reqs ? weight_of(span_of(a, c, r + lane, kRows), hk) : 0;
        int64_t sum = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += up;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + sum > x);
        if (past != 0) {
          const int at = __ffs(past) - 1;
          base += __shfl_sync(0xffffffffu, sum - w, at);
          r += at;
          break;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
        r += 32;
      }
      if (r >= c.num_reqs) return false;  // kv_lens changed under way
      const Span sp = span_of(a, c, r, kRows);
      const int units = units_of(sp);
      const int item = static_cast<int>(div(x - base, units, W * P));
      const int64_t i0 = base + static_cast<int64_t>(item) * units, i1 = i0 + units;
      const int64_t end = x_end < i1 ? x_end : i1;
      const int cost = units - sp.steps;
      const int from = x - i0 > cost ? static_cast<int>(x - i0) - cost : 0;
      const int to = sp.steps > 0 ? static_cast<int>(end - i0) - cost : 0;
      x = end;
      if (sp.steps > 0 && to <= from) continue;  // its steps all lie in another piece
      if (lane == 0) {
        Item it;
        it.r = r;
        it.tile = item / hk;
        it.h = item - it.tile * hk;
        it.rows = min(kRows, sp.n * G - it.tile * kRows);
        it.t0 = sp.t0;
        it.n = sp.n;
        it.len = sp.len;
        it.clipped = sp.clipped;
        it.step = sp.step0 + from;
        it.steps = to - from;
        it.block0 = sp.block0;
        const int64_t room = static_cast<int64_t>(c.max_pages) * (c.page_size / kBlockTokens);
        const int held = (sp.len + kBlockTokens - 1) / kBlockTokens;
        it.block_end = min(static_cast<int>(held < room ? held : room), 2 * (it.step + it.steps));
        const int64_t j0 = sp.steps > 0 ? i0 + cost : i0;
        it.first = static_cast<int>(div((j0 + 1) * P - 1, W, W * P));
        it.pieces = static_cast<int>(div(i1 * P - 1, W, W * P)) - it.first + 1;
        *out = it;
        cursor->x = x;
        cursor->base = base;
        cursor->r = r;
      }
      __syncwarp();
      return true;
    }
    if (lane == 0) cursor->x = x;
    __syncwarp();
    return false;
  };

  // this warp's copies
  const int per_page = c.page_size / kBlockTokens;
  uint32_t phases = 0, armed = 0, present = 0;  // by stage: parity, a copy issued, blocks present (2 bits)
  bool dead = false;                            // a wait gave up: no more copies
  int ahead = 0;                                // steps still to issue
  int blocks_left = 0;                          // of `blocks`, not yet used
  int block = 0;                                // behind blocks_next
  int blocks = -1, blocks_next = -1;            // where the next 32 blocks lie, and the 32 behind them; -1: nowhere
  int stage_in = 0, stage_out = 0;
  const Item* source = items;                   // the item being copied
  auto block_at = [&](int b) {
    if (b < source->block0 || b >= source->block_end) return -1;
    const int col = b / per_page;
    const int64_t page = __ldg(c.block_table + static_cast<int64_t>(source->r) * c.max_pages + col);
    if (page < 0 || page >= c.num_pages) {
      set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
      return -1;
    }
    return static_cast<int>((page * hk + source->h) * per_page + (b - col * per_page));
  };
  auto issue = [&]() {
    if (ahead == 0 || dead) return;
    if (blocks_left == 0) {
      blocks = blocks_next;
      blocks_next = block_at(block + lane);
      block += 32;
      blocks_left = 32;
    }
    const int at = __shfl_sync(0xffffffffu, blocks, 32 - blocks_left + (lane & 1));
    blocks_left -= 2;
    const unsigned mask = __ballot_sync(0xffffffffu, at >= 0) & 3u;
    const uint32_t bar = bar0 + 8 * stage_in;
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(mask) * B::kBytes);
    __syncwarp();
    if (lane < 2 && at >= 0)
      bulk_copy_g2s(smem_u32(ring + stage_in * L::kStage + lane * B::kBytes),
                    c.base + static_cast<int64_t>(at) * B::kBytes, B::kBytes, bar);
    present = (present & ~(3u << (2 * stage_in))) | (mask << (2 * stage_in));
    armed |= 1u << stage_in;
    --ahead;
    if (++stage_in == L::kStages) stage_in = 0;
  };
  auto start = [&](const Item* it) {
    source = it;
    ahead = it->steps;
    if (it->clipped && lane == 0) set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
    block = 2 * it->step;
    blocks = block_at(block + lane);
    blocks_next = block_at(block + 32 + lane);
    block += 64;
    blocks_left = 32;
#pragma unroll 1
    for (int s = 0; s < L::kStages; ++s) issue();
  };

  bool more = next_item(items);
  if (more) start(items);
  rest();
#pragma unroll 1
  for (int which = 0; more; which ^= 1) {
    const Item* const it = items + which;
    const int rows = it->rows;
    // The query rows as B fragments, and what a score needs of each row: the
    // factor that takes it to log2 units, the sum of its elements, its last
    // position, its place in the output.
    uint2 qr[L::kQRegs ? D / 16 : 1];
#pragma unroll 1
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = nt * 8 + g;
      const int flat = it->tile * kRows + rr;
      const int token = flat / G;
      const int64_t head = static_cast<int64_t>(it->h * G + (flat - token * G)) * D;
      const ple_bf16_t* src = a.q + static_cast<int64_t>(it->t0 + token) * a.q_stride + head + j * (D / 4);
      uint4 v[kWords];
      float top = 0.0f;
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        v[w] = make_uint4(0, 0, 0, 0);
        if (rr < rows) v[w] = *reinterpret_cast<const uint4*>(src + 8 * w);
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        float f[8];
        unpack8(v[w], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^k <= top < 2^(k + 1), or below
      const int k = top > 0.0f && top < INFINITY ? max(ilogbf(top), -100) : 0;
      const float down = ldexpf(1.0f, 15 - k);
      float even = 0.0f, odd = 0.0f;  // sums of the elements; the odd ones' are of sixteenths
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        float f[8];
        unpack8(v[w], f);
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float by = i % 2 == 0 ? down : down * 0.0625f;
          p[i] = pack_f16(f[i] * by, f[i + 4] * by);
          const float2 r2 = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
          if (i % 2 == 0) even += r2.x + r2.y;
          else odd += r2.x + r2.y;
        }
        if constexpr (L::kQRegs) {
          qr[2 * w] = make_uint2(p[0], p[1]);
          qr[2 * w + 1] = make_uint2(p[2], p[3]);
        } else {
          qf[((2 * w) * NT + nt) * 32 + lane] = make_uint2(p[0], p[1]);
          qf[((2 * w + 1) * NT + nt) * 32 + lane] = make_uint2(p[2], p[3]);
        }
      }
#pragma unroll
      for (int x2 = 1; x2 < 4; x2 <<= 1) {
        even += __shfl_xor_sync(0xffffffffu, even, x2);
        odd += __shfl_xor_sync(0xffffffffu, odd, x2);
      }
      if (j == 0) {
        // 2^(24 + k - 15) is to come: 2^6 of it with the keys' scales, so that
        // neither is infinite for a row of bf16's largest queries, or keys
        row_info[rr] = ldexpf(a.scale_log2, k + 3);
        row_info[kRows + rr] = ldexpf(fmaf(16.0f, odd, even), -18);
        const int last = a.causal ? it->len - it->n + token : it->len - 1;
        row_last[rr] = rr < rows ? last : -1;
        row_out[rr] = static_cast<int64_t>(it->t0 + token) * a.out_stride + head;
      }
    }
    __syncwarp();
    // positions that every row sees: [all_from, all_to]
    const int all_to = row_last[0];
    const int all_from = a.window > 0 ? max(row_last[rows - 1] - a.window + 1, 0) : 0;

    Results<D, NT> res;
    auto& o = res.o;
    auto& m = res.m;
    auto& l = res.l;  // once the steps are done
    uint64_t l2[NT], off2[NT];  // for two rows: sums of p, and of p (m + 8 s)
    float sum[NT][4];           // of p' (rows 0 and 1 twice)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < D / 16; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][u][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) m[i] = -FLT_MAX;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l2[n] = off2[n] = f2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[n][i] = 0.0f;
    }

    const int p_end = (it->step + it->steps) * kStepTokens;
#pragma unroll 1
    for (int p0 = it->step * kStepTokens; p0 < p_end; p0 += kStepTokens) {
      uint32_t here = 0;
      if (!dead) {
        const bool ok = mbar_try_wait(bar0 + 8 * stage_out, (phases >> stage_out) & 1u) ||
                        mbar_wait(bar0 + 8 * stage_out, (phases >> stage_out) & 1u, nullptr);
        if (__all_sync(0xffffffffu, ok)) {
          here = (present >> (2 * stage_out)) & 3u;
          phases ^= 1u << stage_out;
          armed &= ~(1u << stage_out);
        } else {
          dead = true;
          if (lane == 0) set_dev_err(a.dev_err, PLE_DEVERR_TIMEOUT);
        }
      }
      const uint8_t* st = ring + stage_out * L::kStage;
      const bool masked = here != 3u || p0 < all_from || p0 + kStepTokens - 1 > all_to;
      if (here != 0) {
        const int r0 = g ^ ((g >> 1) & 1);  // token of row g
        float s[NT][2][4];                  // [query tile][block][(token r0, r0 + 8) x (row 2j, 2j + 1)]
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][b][i] = 0.0f;
          const uint8_t* kb = st + b * B::kBytes;
          uint32_t lo[kWords], hi[kWords];
          {
            const uint8_t* p = kb + r0 * B::kRow + j * (D / 8);
            const uint8_t* p8 = p + 8 * B::kRow;
            if constexpr (kWords >= 4) {
#pragma unroll
              for (int w = 0; w < kWords; w += 4) {
                *reinterpret_cast<uint4*>(lo + w) = *reinterpret_cast<const uint4*>(p + 4 * w);
                *reinterpret_cast<uint4*>(hi + w) = *reinterpret_cast<const uint4*>(p8 + 4 * w);
              }
            } else {
              *reinterpret_cast<uint2*>(lo) = *reinterpret_cast<const uint2*>(p);
              *reinterpret_cast<uint2*>(hi) = *reinterpret_cast<const uint2*>(p8);
            }
          }
#pragma unroll
          for (int w = 0; w < kWords; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0 = code_bits(lo[w], 2 * h), a1 = code_bits(hi[w], 2 * h);
              const uint32_t a2 = code_bits(lo[w], 2 * h + 1), a3 = code_bits(hi[w], 2 * h + 1);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                uint2 f;
                if constexpr (L::kQRegs) f = qr[(2 * w + h) * NT + n];
                else f = qf[((2 * w + h) * NT + n) * 32 + lane];
                mma_f16(s[n][b], a0, a1, a2, a3, f.x, f.y);
              }
            }
        }
        // scores in units of log2: scale and offset, then the mask; two rows at a time
        float vs[2][2], vm[2][2];  // the values' scale, and offset + 8 scales
        uint32_t unseen = 0;       // bit (query tile, block, token, row)
        float most = 0.0f;         // of the scales that the lane's rows see
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = r0 + 8 * e;
            const uint32_t kp = bf2_mul(*reinterpret_cast<const uint32_t*>(st + b * B::kBytes + B::kPairs + tok * 4),
                                        0x3F804280u);  // the scale times 2^6
            const uint32_t vp = *reinterpret_cast<const uint32_t*>(st + b * B::kBytes + B::kVPairs + tok * 4);
            const uint64_t ks = f2(bf_lo(kp), bf_lo(kp)), km = f2(bf_hi(kp), bf_hi(kp));
            vs[b][e] = bf_lo(vp);
            vm[b][e] = fmaf(8.0f, bf_lo(vp), bf_hi(vp));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint64_t f = *reinterpret_cast<const uint64_t*>(row_info + n * 8 + 2 * j);
              const uint64_t sq = *reinterpret_cast<const uint64_t*>(row_info + kRows + n * 8 + 2 * j);
              const uint64_t z = f2_mul(f, f2_fma(ks, f2(s[n][b][2 * e], s[n][b][2 * e + 1]), f2_mul(km, sq)));
              f2_split(z, s[n][b][2 * e], s[n][b][2 * e + 1]);
            }
            if (masked) {
              const int p = p0 + b * kBlockTokens + tok;
              const bool there = (here >> b) & 1u;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const int2 lasts = *reinterpret_cast<const int2*>(row_last + n * 8 + 2 * j);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int last = i == 0 ? lasts.x : lasts.y;
                  if (!there || p > last || (a.window > 0 && p <= last - a.window)) {
                    s[n][b][2 * e + i] = -INFINITY;
                    unseen |= 1u << (n * 8 + b * 4 + e * 2 + i);
                  }
                }
              }
              constexpr uint32_t kRowBits = 0x03030303u >> (8 * (4 - NT));
              if ((~unseen & (kRowBits << (b * 4 + e * 2))) != 0) most = fmaxf(most, fabsf(vs[b][e]));
            } else {
              most = fmaxf(most, fabsf(vs[b][e]));
            }
          }
        // The running maximum is raised only when a score passes it by 2^6:
        // weights of up to 64 cost no precision in float32 or f16, and a
        // step without a raise needs no exchange between lanes.
        bool raise = false;
        float top[2 * NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float t = fmaxf(fmaxf(s[n][0][i], s[n][0][2 + i]), fmaxf(s[n][1][i], s[n][1][2 + i]));
            top[2 * n + i] = t;
            raise |= t > m[2 * n + i] + 6.0f;
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i) {
            float t = top[i];
#pragma unroll
            for (int x2 = 4; x2 < 32; x2 <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x2));
            const float next = fmaxf(m[i], t);
            const float keep = ex2(m[i] - next);
            m[i] = next;
            const int n = i / 2, e = i & 1;
            float la, lb;
            f2_split(l2[n], la, lb);
            l2[n] = e == 0 ? f2(la * keep, lb) : f2(la, lb * keep);
            f2_split(off2[n], la, lb);
            off2[n] = e == 0 ? f2(la * keep, lb) : f2(la, lb * keep);
            sum[n][e] *= keep;
#pragma unroll
            for (int u = 0; u < D / 16; ++u) { o[n][u][e] *= keep; o[n][u][2 + e] *= keep; }
          }
        }
        const bool wide = __any_sync(0xffffffffu, !(most < 1024.0f) || (most < 0x1p-9f && most > 0.0f));
        uint32_t pt[NT][2][2];  // weights times the values' scale as B fragments: f16, or bf16 times 2^-6
        auto weights = [&](auto with_mask) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float by = wide ? vs[b][e] * 0x1p-6f : vs[b][e];
              const uint64_t by2 = f2(by, by), vm2 = f2(vm[b][e], vm[b][e]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float p[2], w[2];
                f2_split(f2_add(f2(s[n][b][2 * e], s[n][b][2 * e + 1]), f2(-m[2 * n], -m[2 * n + 1])), p[0], p[1]);
                p[0] = ex2(p[0]);
                p[1] = ex2(p[1]);
                const uint64_t p2 = f2(p[0], p[1]);
                l2[n] = f2_add(l2[n], p2);
                f2_split(f2_mul(p2, by2), w[0], w[1]);
                uint64_t next = f2_fma(p2, vm2, off2[n]);
                if constexpr (decltype(with_mask)::value) {
                  // a value that is not seen meets no weight, not even zero: it may be NaN
                  float was[2], now[2];
                  f2_split(off2[n], was[0], was[1]);
                  f2_split(next, now[0], now[1]);
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if ((unseen >> (n * 8 + b * 4 + e * 2 + i)) & 1u) { now[i] = was[i]; w[i] = 0.0f; }
                  next = f2(now[0], now[1]);
                }
                off2[n] = next;
                pt[n][b][e] = transpose8x8(wide ? pack2(w[0], w[1]) : pack_f16(w[0], w[1]));
              }
            }
        };
        if (masked) weights(std::true_type{});
        else weights(std::false_type{});
        auto values = [&](auto in_bf16) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint8_t* vb = st + b * B::kBytes + B::kV + g * (D / 16);
          uint32_t v[4][kVWords];  // tokens 2j, 2j + 1, 2j + 8, 2j + 9 in the rows' order
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 2 * j + (i & 1);
            const uint8_t* p = vb + ((row ^ ((row >> 1) & 1)) + 8 * (i >> 1)) * B::kRow;
            if constexpr (kVWords == 4) *reinterpret_cast<uint4*>(v[i]) = *reinterpret_cast<const uint4*>(p);
            else if constexpr (kVWords == 2) *reinterpret_cast<uint2*>(v[i]) = *reinterpret_cast<const uint2*>(p);
            else v[i][0] = *reinterpret_cast<const uint32_t*>(p);
          }
          constexpr bool kBf16 = decltype(in_bf16)::value;
          constexpr uint32_t kOne = kBf16 ? 0x42804280u : 0x3C003C00u;  // 2^6, or 1
          auto product = [](float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
            if constexpr (kBf16) mma_bf16(c, a0, a1, a2, a3, b0, b1);
            else mma_f16(c, a0, a1, a2, a3, b0, b1);
          };
#pragma unroll
          for (int n = 0; n < NT; ++n) product(sum[n], kOne, kOne, kOne, kOne, pt[n][b][0], pt[n][b][1]);
          auto code = [](uint32_t x, int i) { return kBf16 ? times_2_115(code_bits(x, i)) : code_bits(x, i); };
#pragma unroll
          for (int w = 0; w < kVWords; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const unsigned sel = half == 0 ? 0x5410u : 0x7632u;
              const uint32_t x0 = __byte_perm(v[0][w], v[1][w], sel), x1 = __byte_perm(v[2][w], v[3][w], sel);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t a0 = code(x0, 2 * k), a1 = code(x0, 2 * k + 1);
                const uint32_t a2 = code(x1, 2 * k), a3 = code(x1, 2 * k + 1);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  product(o[n][w * 4 + half * 2 + k], a0, a1, a2, a3, pt[n][b][0], pt[n][b][1]);
              }
            }
        }
        };
        if (wide) values(std::true_type{});
        else values(std::false_type{});
      }
      __syncwarp();  // every lane has read the stage
      if (++stage_out == L::kStages) stage_out = 0;
      issue();
    }

    // the next item's copies fly while this one's results are written
    more = next_item(items + (which ^ 1));
    if (more) start(items + (which ^ 1));

#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float off[2];
      f2_split(l2[n], l[2 * n], l[2 * n + 1]);
      f2_split(off2[n], off[0], off[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          l[2 * n + e] += __shfl_xor_sync(0xffffffffu, l[2 * n + e], sh);
          off[e] += __shfl_xor_sync(0xffffffffu, off[e], sh);
        }
        off[e] = fmaf(-8.0f, sum[n][e], off[e]);
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {
          o[n][u][e] = fmaf(0x1p24f, o[n][u][e], off[e]);
          o[n][u][2 + e] = fmaf(0x1p20f, o[n][u][2 + e], off[e]);
        }
      }
    }
    const int first = it->first;
    int count = it->pieces;  // of this level
    if (count > 1) {
      store_partial<D, NT>(res, partial + static_cast<int64_t>(slot_of(first, piece - first)) * L::kSlot);
      // level by level: the last to arrive in a group of kFan goes on for it
      unsigned* counter = counters;
      int k = piece - first, stride = 1;
      for (;;) {
        const int lead = k / kFan * kFan;  // of the group, in units of stride
        const int members = min(kFan, count - lead);
        __threadfence();
        __syncwarp();
        unsigned before = 0;
        if (lane == 0) {
          unsigned* at = counter + slot_of(first, lead * stride);
          before = atomicAdd(at, 1u);
          if (before == static_cast<unsigned>(members - 1)) *at = 0;
        }
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before != static_cast<unsigned>(members - 1)) break;
        __threadfence();
        load_joined<D, NT>(res, partial, first, lead * stride, stride, members);
        if (count <= kFan) {
          count = 1;
          break;
        }
        __syncwarp();  // every lane has read what is written over
        store_partial<D, NT>(res, partial + static_cast<int64_t>(slot_of(first, lead * stride)) * L::kSlot);
        k /= kFan;
        count = (count + kFan - 1) / kFan;
        stride *= kFan;
        counter += 2 * gridDim.x * kWarps;
      }
    }
    if (count == 1) store_out<D, NT>(res, a.out, row_out, rows);
    __syncwarp();  // row_info and the item are free
  }
  // never leave with a copy in flight
  for (int s = 0; s < L::kStages; ++s)
    if ((armed >> s) & 1u) mbar_wait(bar0 + 8 * s, (phases >> s) & 1u, nullptr);
}

// From how many rows (query tokens times heads of a group) on a request's
// cache is read for 256 rows at a time, by the 5th-generation tensor cores.
// This file's kernel takes up to 32 rows in one pass over the cache and is
// bound by the cache's bytes; the other's time does not depend on the rows up
// to 256 and is bound by turning codes into operands. Measured at 8 kv heads,
// 2048 positions unless stated, this kernel / the other, us:
//   16 rows,  4 requests  28 /  26;  1 request, 64k positions  52 /  82
//   32 rows,  4 requests  48 /  30;  1 request, 64k positions  91 /  91
//            16 requests  62 /  47;  32 requests  77 / 95;  64 requests  128 / 185
//   48 rows, 16 requests  69 /  47;  32 requests 112 / 95;  64 requests  228 / 186
// So 33 rows always go to the other, and 17 to 32 do where a CTA for each
// request and kv head finds an SM of its own. Heads of 256 (16 rows a pass
// here, half the buffers there) meet later; 2 kv heads:
//   64 rows,  1 request  37 / 43;  64 requests  89 / 86
//  128 rows,  1 request  38 / 45;  64 requests 154 / 90
int many_rows(int num_reqs, int num_kv_heads, int head_dim) {
  return head_dim == 256 ? 96 : int64_t(num_reqs) * num_kv_heads <= num_sms() ? 17 : 33;
}

constexpr int kMaxWarps = 16;  // of an SM, of any variant
constexpr int kLevels = 4;   // of joining: more than 8^4 warps there are not

// Arrivals, by level and slot.
size_t counter_bytes() { return size_t(kLevels) * 2 * num_sms() * kMaxWarps * 4 / 256 * 256 + 256; }

template <int D, int NT>
size_t partial_bytes() {
  return size_t(2) * num_sms() * Split<D, NT>::kWarps * Split<D, NT>::kSlot * 4;
}

// Counters, then two partial results a piece of the variant that needs most.
size_t workspace_bytes_of(int head_dim) {
  size_t n = 0;
  if (head_dim == 64) n = std::max(partial_bytes<64, 1>(), std::max(partial_bytes<64, 2>(), partial_bytes<64, 4>()));
  if (head_dim == 128) n = std::max(partial_bytes<128, 1>(), std::max(partial_bytes<128, 2>(), partial_bytes<128, 4>()));
  if (head_dim == 256) n = std::max(partial_bytes<256, 1>(), partial_bytes<256, 2>());
  return counter_bytes() + (n + 255) / 256 * 256;
}

template <int D, int NT>
cudaError_t launch_split(const AttentionArgs& a, const KvCache& c, unsigned* counters, float* partial,
                         cudaStream_t stream) {
  using L = Split<D, NT>;
  const auto kernel = attention_split_kernel<D, NT>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (err != cudaSuccess) return err;
  return launch_kernel(kernel, dim3(num_sms()), dim3(L::kWarps * 32), L::kSmem, stream, 1, a, c,
                       counters, partial);
}

}  // namespace
}  // namespace ple

using namespace ple;

PLE_EXPORT size_t ple_kv_attention_workspace(int32_t num_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 || ple_kv_block_bytes(head_dim) == 0)
    return 0;
  return workspace_bytes_of(head_dim);
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
  // query rows are 32-bit in the kernel, and so are block numbers in the kernel (2^31 blocks would be a cache of terabytes)
  if (num_pages > 0 && num_pages > (int64_t(1) << 31) / num_kv_heads / (page_size / kBlockTokens))
    return fail(PLE_ERR_UNSUPPORTED, "%s: %lld pages", name, static_cast<long long>(num_pages));
  if (num_heads > 0 && num_tokens > INT32_MAX / 2 / num_heads)
    return fail(PLE_ERR_UNSUPPORTED, "%s: %lld tokens of %d heads", name, static_cast<long long>(num_tokens), num_heads);
  if (num_heads < 1 || num_heads % num_kv_heads != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: %d heads over %d kv heads", name, num_heads, num_kv_heads);
  if (q == nullptr || out == nullptr || !aligned16(q) || !aligned16(out) || q_stride % 8 != 0 || out_stride % 8 != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned, their strides multiples of 8", name);
  const int64_t row = int64_t(num_heads) * head_dim * 2;
  if (!(q == out && q_stride == out_stride) &&
      rows_overlap({out, num_tokens, out_stride * 2, row}, {q, num_tokens, q_stride * 2, row}))
    return fail(PLE_ERR_INVALID_ARG, "%s: out overlaps q without being it", name);
  if (!(scale > 0.0f) || !std::isfinite(scale))
    return fail(PLE_ERR_INVALID_ARG, "%s: scale %g", name, scale);
  if (max_query_len < 0 || window < 0 || (window > 0 && !causal))
    return fail(PLE_ERR_INVALID_ARG, "%s: max_query_len %d, window %d%s", name, max_query_len, window,
                causal ? "" : " without causal");
  const size_t need = ple_kv_attention_workspace(num_heads, num_kv_heads, head_dim);
  if (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: workspace of %zu bytes, 256-byte aligned, needed", name, need);
  // the rows of a request and kv head, at most
  const int64_t tokens = max_query_len > 0 && max_query_len < num_tokens ? max_query_len : num_tokens;
  const int64_t rows = tokens * (num_heads / num_kv_heads);
  const int many = many_rows(num_reqs, num_kv_heads, head_dim);
  // a hint that is too small must lose no rows: without the other kernel this one takes them all
  const AttentionArgs a{q, q_stride, num_tokens, num_heads, scale * 1.4426950408889634f, causal != 0,
                        window, out, out_stride, dev_err, rows >= many ? many : INT32_MAX};
  const KvCache c{const_cast<uint8_t*>(static_cast<const uint8_t*>(cache)), num_pages, page_size,
                  num_kv_heads, block_table, max_pages, query_start_loc, num_reqs, kv_lens};
  unsigned* counters = static_cast<unsigned*>(workspace);
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + counter_bytes());
  cudaError_t err = cudaSuccess;
  // both kernels' partial results may lie in one place: one runs after the other
  if (rows >= many) err = launch_prefill(a, c, head_dim, partial, need - counter_bytes(), stream);
  if (err != cudaSuccess) return check_cuda(err, name);
  if (head_dim == 64)
    err = rows <= 8 ? launch_split<64, 1>(a, c, counters, partial, stream)
        : rows <= 16 ? launch_split<64, 2>(a, c, counters, partial, stream)
                     : launch_split<64, 4>(a, c, counters, partial, stream);
  else if (head_dim == 128)
    err = rows <= 8 ? launch_split<128, 1>(a, c, counters, partial, stream)
        : rows <= 16 ? launch_split<128, 2>(a, c, counters, partial, stream)
                     : launch_split<128, 4>(a, c, counters, partial, stream);
  else
    err = rows <= 8 ? launch_split<256, 1>(a, c, counters, partial, stream)
                    : launch_split<256, 2>(a, c, counters, partial, stream);
  return check_cuda(err, name);
}
