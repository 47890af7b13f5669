// ple_kv_attention: grouped-query attention over the paged 4-bit cache.
#include "kv_cache.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

namespace ple {
namespace {

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

// ---------------------------------------------------------------------------
// Few query rows: the cache split over the card
// ---------------------------------------------------------------------------
// Work. An item is (request, tile of 8 NT query rows, kv head); its cost is
// the number of 32-token steps of the cache it reads. The steps of all items
// lie on one line, cut into equal pieces, one for each CTA, so a single long
// request and hundreds of ragged ones load the card alike. An item that a cut
// falls into leaves partial results (row maxima, sums, unnormalised outputs)
// in the workspace, and the CTA that arrives last joins them in the order of
// the pieces: results do not depend on timing. Every CTA finds its piece from
// query_start_loc and kv_lens itself: one launch, no plan on the host.
//
// Streams. Each of a CTA's four warps has its own share of the piece's
// steps and its own ring of stages in shared memory; a stage is two cache
// blocks, each one bulk copy. No warp waits for another until the item ends,
// and the next item's first copies fly while this one's results are joined.
//
// Products, on warp-wide matrix instructions (16 x 8 x 16, f32 sums; reading
// the cache and unpacking it, not their rate, is the bound):
//   S^T = K Q^T     16 tokens x 8 query rows, f16
//   O^T = V^T P^T   16 elements x 8 query rows, bf16
// so that a group of up to 8 query heads fills a tile, and the codes are the
// A operand of both. Unpacking a word of 8 codes:
//   Masked out where they stand, a byte's codes are subnormal numbers that no
//   bit has to be added to: bits 0-3 of a half are c 2^-24 as f16 (c 2^-133
//   as bf16), bits 4-7 sixteen times that. So a word of eight codes takes
//   four masks and one shift by a byte.
//   K: f16 subnormals multiply as they are; the query elements that meet the
//     second kind are divided by 16, and 2^24 goes into the rows' factors.
//   V: one fused multiply-add makes bf16 (c - 8) / 64 or (c - 8) / 4, so that
//     sums over long caches hold no offset; 64 and 4 are taken out at the end.
// Query rows are scaled to [1, 2) by a power of two each, which keeps f16
// exact for bf16 queries (elements below 2^-14 of the row's largest round at
// 2^-24 of it). Scale and offset of a token meet the float32 sums instead of
// its elements:
//   <q, K_t> = s_t sum_d q_d c_td + m_t sum_d q_d
//   sum_t p_t V_t = sum_t p'_t (c_t - 8) + sum_t p_t (m_t + 8 s_t),  p' = bf16(p s)
// p' is the only rounding to fewer bits, and it meets codes centred on 8, so
// that an offset far from zero costs no precision.
// The contraction index of a product may run in any order: a lane's 16 bytes
// of a K row are 32 neighbouring elements, and the query's fragments follow
// that order; two tokens' V bytes are interleaved with one permute a word.
// Token rows are taken in the order t ^ (t >> 1 & 1), which lets the V loads
// of neighbouring lanes fall on different banks.
constexpr int kWarps = 4;
constexpr int kStepTokens = 2 * kBlockTokens;

// NT tiles of 8 query rows a warp; registers and shared memory set the CTAs an SM holds.
template <int D, int NT>
struct Split {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStage = 2 * KvBlock<D>::kBytes;
  static constexpr int kCtas = D == 256 || NT == 4 ? 2 : NT == 2 ? 3 : 4;  // per SM
  static constexpr int kStages = D == 256 ? 2 : D == 64 || NT == 4 ? 4 : NT == 2 ? 3 : 2;
  static constexpr bool kQRegs = NT * D <= 256;      // query fragments in registers
  static constexpr int kPass = 8;                    // rows joined at a time
  static constexpr int kGroup = D / 8 + 2;           // a lane group's elements, padded
  static constexpr int kPitch = 8 * kGroup + 4;      // floats of a row in the joining buffer
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kFrags = NT * (D / 16) * 32 * 8;  // bytes of query fragments
  static constexpr int kJoin = kWarps * kPass * kPitch * 4;
  static constexpr int kMl = kWarps * kRows * 8;
  static constexpr int kRowInfo = kRows * 24;        // a query row's factor, sum, last position, place in the output
  static constexpr int kSegments = 2 * 128;  // the present and the next segment
  static constexpr int kSmem = kRing + kFrags + kJoin + kMl + kRowInfo + kSegments + kWarps * kStages * 8 + 16;
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Codes i and i + 4 of a word (i = 0..3) as f16 pair: c 2^-24 for even i,
// c 2^-20 for odd i.
__device__ __forceinline__ uint32_t k_pair(uint32_t word, int i) {
  return (i < 2 ? word : word >> 8) & (i % 2 == 0 ? 0x000F000Fu : 0x00F000F0u);
}

// Codes i of the two halves of a word (i = 0..3) as bf16 pair: (c - 8) / 64
// for even i, (c - 8) / 4 for odd i.
__device__ __forceinline__ uint32_t v_pair(uint32_t word, int i) {
  uint32_t y;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(k_pair(word, i)), "r"(0x7F007F00u) /* 2^127 */,
      "r"(i % 2 == 0 ? 0xBE00BE00u /* -1/8 */ : 0xC000C000u /* -2 */));
  return y;
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
  s.tiles = (s.n * (a.num_heads / c.num_kv_heads) + tile_rows - 1) / tile_rows;
  return s;
}

// An item's length on the line: what starting and joining it costs, in steps,
// then its steps; 1 for an item that only writes zeros.
constexpr int kItemCost = 4;
__device__ __forceinline__ int units_of(const Span& s) { return s.steps > 0 ? kItemCost + s.steps : 1; }

__device__ __forceinline__ int64_t weight_of(const Span& s, int hk) {
  return static_cast<int64_t>(s.tiles) * hk * units_of(s);
}

// A CTA's share of one item.
struct Segment {
  Span s;
  int64_t end;        // where the request's items end on the line
  int r, tile, h, rows;
  int from, to;       // steps, relative to s.step0
  int pieces, first;  // CTAs that share the item's steps, the first of them
};

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, (Split<D, NT>::kCtas))
attention_split_kernel(const AttentionArgs a, const KvCache c, unsigned* __restrict__ counters,
                       float* __restrict__ partial) {
  using L = Split<D, NT>;
  using B = KvBlock<D>;
  constexpr int kRows = L::kRows;
  constexpr int kWords = D / 32;   // K words of a lane and token
  constexpr int kVWords = D / 64;  // V words of a lane and token
  extern __shared__ __align__(128) uint8_t smem[];
  uint2* qf = reinterpret_cast<uint2*>(smem + L::kRing);
  float* join = reinterpret_cast<float*>(smem + L::kRing + L::kFrags);
  float2* ml = reinterpret_cast<float2*>(smem + L::kRing + L::kFrags + L::kJoin);
  // for each query row: factor to log2 units, sum, last position, place in the output
  float* row_info = reinterpret_cast<float*>(smem + L::kRing + L::kFrags + L::kJoin + L::kMl);
  Segment* segments = reinterpret_cast<Segment*>(smem + L::kRing + L::kFrags + L::kJoin + L::kMl + L::kRowInfo);
  const int* row_last = reinterpret_cast<const int*>(row_info + 2 * kRows);
  int64_t* row_out = reinterpret_cast<int64_t*>(row_info + 4 * kRows);
  static_assert(sizeof(Segment) <= 128, "two segments a warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int g = lane >> 2, j = lane & 3;
  uint8_t* ring = smem + warp * L::kStages * L::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kSmem - 16 - kWarps * L::kStages * 8);
  const uint32_t bar0 = smem_u32(bars + warp * L::kStages);
  int64_t* total = reinterpret_cast<int64_t*>(smem + L::kSmem - 16);
  int* last_flag = reinterpret_cast<int*>(smem + L::kSmem - 8);

  if (lane == 0) {
    for (int s = 0; s < L::kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == 0) *total = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int G = a.num_heads / c.num_kv_heads;
  const int hk = c.num_kv_heads;
  // all items' steps
  {
    int64_t mine = 0;
    for (int r = threadIdx.x; r < c.num_reqs; r += kWarps * 32) mine += weight_of(span_of(a, c, r, kRows), hk);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0 && mine > 0) atomicAdd(reinterpret_cast<unsigned long long*>(total), static_cast<unsigned long long>(mine));
    for (int64_t i = int64_t(blockIdx.x) * (kWarps * 32) + threadIdx.x; i < c.num_reqs; i += int64_t(gridDim.x) * (kWarps * 32))
      check_qsl(c.qsl, c.num_reqs, a.T, i, a.dev_err);
    // padding tokens' rows
    int64_t pad = __ldg(c.qsl + c.num_reqs);
    pad = pad < 0 ? 0 : pad;
    const int64_t vecs = static_cast<int64_t>(a.num_heads) * (D / 8);
    for (int64_t i = pad * vecs + int64_t(blockIdx.x) * (kWarps * 32) + threadIdx.x; i < a.T * vecs;
         i += int64_t(gridDim.x) * (kWarps * 32))
      *reinterpret_cast<uint4*>(a.out + i / vecs * a.out_stride + i % vecs * 8) = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  const int64_t W = *total;
  // pieces of at least one step for each warp
  const int64_t most = (W + kWarps + kItemCost - 1) / (kWarps + kItemCost);
  const int64_t S = most < gridDim.x ? most : gridDim.x;
  if (blockIdx.x >= S) return;
  int64_t x = blockIdx.x * W / S;
  const int64_t x_end = (blockIdx.x + 1) * W / S;

  // the request that x lies in; base: its first step on the line
  int r = 0;
  int64_t base = 0;
  auto seek = [&]() {  // from request r at base on, the first request that ends past x
    for (;;) {
      int64_t w = r + lane < c.num_reqs ? weight_of(span_of(a, c, r + lane, kRows), hk) : 0;
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
        return;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
      r += 32;
      if (r >= c.num_reqs) return;  // not reached: x < W
    }
  };

  // The next segment with something to do, from x on; false if there is none.
  // Every warp finds it for itself and writes the same values down.
  auto next_segment = [&](Segment* out) {
    while (x < x_end) {
      const Span sp = span_of(a, c, r, kRows);
      const int units = units_of(sp);
      const int64_t end = base + static_cast<int64_t>(sp.tiles) * hk * units;
      if (x >= end) {
        base = end;
        ++r;
        seek();
        continue;
      }
      const int item = static_cast<int>((x - base) / units);
      const int64_t i0 = base + static_cast<int64_t>(item) * units, i1 = i0 + units;
      const int64_t to = x_end < i1 ? x_end : i1;
      const int cost = units - sp.steps;
      const int from = x - i0 > cost ? static_cast<int>(x - i0) - cost : 0;
      const int upto = static_cast<int>(to - i0) - cost;
      x = to;
      if (sp.steps > 0 && upto <= from) continue;  // the item's steps are all another CTA's
      if (lane == 0) {
        Segment q;
        q.s = sp;
        q.end = end;
        q.r = r;
        q.tile = item / hk;
        q.h = item - q.tile * hk;
        q.rows = min(kRows, sp.n * G - q.tile * kRows);
        q.from = from;
        q.to = sp.steps > 0 ? upto : from;
        const int64_t j0 = sp.steps > 0 ? i0 + cost : i0;
        q.first = static_cast<int>(((j0 + 1) * S - 1) / W);
        q.pieces = static_cast<int>((i1 * S - 1) / W) - q.first + 1;
        *out = q;
      }
      __syncwarp();
      return true;
    }
    return false;
  };

  // this warp's copies
  const int per_page = c.page_size / kBlockTokens;
  uint32_t phases = 0, armed = 0, present = 0;  // by stage: parity, a copy issued, blocks present (2 bits)
  bool dead = false;                            // a wait gave up: no more copies
  int issue_step = 0, issue_end = 0;            // absolute steps
  int pages_at = 0;                             // first block of `blocks`
  int blocks = -1, blocks_next = -1;            // where request blocks pages_at + lane and + 32 lie; -1: nowhere
  const int32_t* table = c.block_table;
  int block_begin = 0, block_end = 0;           // blocks that this warp's rows may see
  int issue_h = 0;
  int stage_in = 0, stage_out = 0;
  auto block_at = [&](int block) {
    if (block < block_begin || block >= block_end) return -1;
    const int col = block / per_page;
    const int64_t page = __ldg(table + col);
    if (page < 0 || page >= c.num_pages) {
      set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
      return -1;
    }
    return static_cast<int>((page * hk + issue_h) * per_page + (block - col * per_page));
  };
  auto issue = [&]() {
    if (issue_step >= issue_end || dead) return;
    const int b = 2 * issue_step - pages_at;
    const int at = __shfl_sync(0xffffffffu, blocks, b + (lane & 1));
    const unsigned mask = __ballot_sync(0xffffffffu, at >= 0) & 3u;
    const uint32_t bar = bar0 + 8 * stage_in;
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(mask) * B::kBytes);
    __syncwarp();
    if (lane < 2 && at >= 0)
      bulk_copy_g2s(smem_u32(ring + stage_in * L::kStage + lane * B::kBytes),
                    c.base + static_cast<int64_t>(at) * B::kBytes, B::kBytes, bar);
    if (b == 30) {
      pages_at += 32;
      blocks = blocks_next;
      blocks_next = block_at(pages_at + 32 + lane);
    }
    present = (present & ~(3u << (2 * stage_in))) | (mask << (2 * stage_in));
    armed |= 1u << stage_in;
    ++issue_step;
    if (++stage_in == L::kStages) stage_in = 0;
  };
  auto share = [&](const Segment& q, int& from, int& to) {  // of this warp
    const int per = (q.to - q.from + kWarps - 1) / kWarps;
    from = min(q.from + warp * per, q.to);
    to = min(from + per, q.to);
  };
  auto start = [&](const Segment& q) {
    int from, to;
    share(q, from, to);
    issue_step = q.s.step0 + from;
    issue_end = q.s.step0 + to;
    issue_h = q.h;
    table = c.block_table + static_cast<int64_t>(q.r) * c.max_pages;
    const int64_t room = static_cast<int64_t>(c.max_pages) * per_page;
    const int64_t held = (q.s.len + kBlockTokens - 1) / kBlockTokens;
    block_end = static_cast<int>(held < room ? held : room);
    block_begin = q.s.block0;
    // not past this warp's own steps: what it never reads raises no flag
    block_end = min(block_end, 2 * issue_end);
    if (q.s.clipped && lane == 0) set_dev_err(a.dev_err, PLE_DEVERR_BOUNDS);
    pages_at = 2 * issue_step;
    blocks = block_at(pages_at + lane);
    blocks_next = block_at(pages_at + 32 + lane);
#pragma unroll 1
    for (int s = 0; s < L::kStages; ++s) issue();
  };

  seek();
  if (!next_segment(segments)) return;
  start(segments[0]);
  for (int which = 0;; which ^= 1) {
    const Segment& q = segments[which];
    // the tile's query rows as B fragments, and what a score needs of them
    const int rows = q.rows;
    for (int nt = warp; nt < NT; nt += kWarps) {
      const int rr = nt * 8 + g;
      const int flat = q.tile * kRows + rr;
      const int token = flat / G;
      const int64_t head = static_cast<int64_t>(q.h * G + (flat - token * G)) * D;
      const ple_bf16_t* src = a.q + static_cast<int64_t>(q.s.t0 + token) * a.q_stride + head + j * (D / 4);
      uint4 v[kWords];
      float top = 0.0f;
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        v[w] = make_uint4(0, 0, 0, 0);
        if (rr < rows) v[w] = *reinterpret_cast<const uint4*>(src + 8 * w);
        float f[8];
        unpack8(v[w], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^k <= top < 2^(k + 1)
      const int k = top > 0.0f && top < INFINITY ? max(ilogbf(top), -126) : 0;
      const float down = ldexpf(1.0f, -k);
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
        qf[((2 * w) * NT + nt) * 32 + lane] = make_uint2(p[0], p[1]);
        qf[((2 * w + 1) * NT + nt) * 32 + lane] = make_uint2(p[2], p[3]);
      }
#pragma unroll
      for (int x2 = 1; x2 < 4; x2 <<= 1) {
        even += __shfl_xor_sync(0xffffffffu, even, x2);
        odd += __shfl_xor_sync(0xffffffffu, odd, x2);
      }
      if (j == 0) {
        row_info[rr] = ldexpf(a.scale_log2, k + 24);
        row_info[kRows + rr] = ldexpf(fmaf(16.0f, odd, even), -24);
        const int last = a.causal ? q.s.len - q.s.n + token : q.s.len - 1;
        reinterpret_cast<int*>(row_info)[2 * kRows + rr] = rr < rows ? last : -1;
        row_out[rr] = static_cast<int64_t>(q.s.t0 + token) * a.out_stride + head;
      }
    }
    __syncthreads();
    uint2 qr[L::kQRegs ? NT * (D / 16) : 1];
    if constexpr (L::kQRegs) {
#pragma unroll
      for (int i = 0; i < NT * (D / 16); ++i) qr[i] = qf[i * 32 + lane];
    }
    // positions that every row of the tile sees: [all_from, all_to]
    int all_from = 0, all_to;
    {
      const int last0 = row_last[0], last1 = row_last[rows - 1];
      all_to = last0;
      if (a.window > 0) all_from = max(last1 - a.window + 1, 0);
    }

    float o[NT][D / 16][4];
    float m[2 * NT], l[2 * NT], off[2 * NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < D / 16; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][u][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) { m[i] = -FLT_MAX; l[i] = 0.0f; off[i] = 0.0f; }
    const int step0 = q.s.step0;

    int from, to;
    share(q, from, to);
#pragma unroll 1
    for (int step = from; step < to; ++step) {
      const int p0 = (step0 + step) * kStepTokens;
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
              const uint32_t a0 = k_pair(lo[w], 2 * h), a1 = k_pair(hi[w], 2 * h);
              const uint32_t a2 = k_pair(lo[w], 2 * h + 1), a3 = k_pair(hi[w], 2 * h + 1);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                uint2 f;
                if constexpr (L::kQRegs) f = qr[(2 * w + h) * NT + n];
                else f = qf[((2 * w + h) * NT + n) * 32 + lane];
                mma_f16(s[n][b], a0, a1, a2, a3, f.x, f.y);
              }
            }
        }
        // scores in units of log2: scale and offset, then the mask
        float vs[2][2], vm[2][2];  // the values' scale, and offset + 8 scales
        uint32_t unseen = 0;       // bit (query tile, block, token, row)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = r0 + 8 * e;
            const uint32_t kp = *reinterpret_cast<const uint32_t*>(st + b * B::kBytes + B::kPairs + tok * 4);
            const uint32_t vp = *reinterpret_cast<const uint32_t*>(st + b * B::kBytes + B::kVPairs + tok * 4);
            const float ks = bf_lo(kp), km = bf_hi(kp);
            vs[b][e] = bf_lo(vp);
            vm[b][e] = fmaf(8.0f, bf_lo(vp), bf_hi(vp));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float2 f = *reinterpret_cast<const float2*>(row_info + n * 8 + 2 * j);
              const float2 sq = *reinterpret_cast<const float2*>(row_info + kRows + n * 8 + 2 * j);
              s[n][b][2 * e] = f.x * fmaf(ks, s[n][b][2 * e], km * sq.x);
              s[n][b][2 * e + 1] = f.y * fmaf(ks, s[n][b][2 * e + 1], km * sq.y);
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
            }
          }
        // The running maximum is raised only when a score passes it by 2^8:
        // weights of up to 256 cost no precision in float32 or bf16, and a
        // step without a raise needs no exchange between lanes.
        bool raise = false;
        float top[2 * NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float t = fmaxf(fmaxf(s[n][0][i], s[n][0][2 + i]), fmaxf(s[n][1][i], s[n][1][2 + i]));
            top[2 * n + i] = t;
            raise |= t > m[2 * n + i] + 8.0f;
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
            l[i] *= keep;
            off[i] *= keep;
            const int n = i / 2, e = i & 1;
#pragma unroll
            for (int u = 0; u < D / 16; ++u) { o[n][u][e] *= keep; o[n][u][2 + e] *= keep; }
          }
        }
        uint32_t pt[NT][2][2];  // weights times the values' scale, bf16, as B fragments
        auto weights = [&](auto with_mask) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float p = ex2(s[n][b][2 * e + i] - m[2 * n + i]);
                  l[2 * n + i] += p;
                  w[i] = p * vs[b][e];
                  const float next = fmaf(p, vm[b][e], off[2 * n + i]);
                  // a value that is not seen meets no weight, not even zero: it may be NaN
                  const bool skip = decltype(with_mask)::value && ((unseen >> (n * 8 + b * 4 + e * 2 + i)) & 1u);
                  off[2 * n + i] = skip ? off[2 * n + i] : next;
                  w[i] = skip ? 0.0f : w[i];
                }
                pt[n][b][e] = transpose8x8(pack2(w[0], w[1]));
              }
        };
        if (masked) weights(std::true_type{});
        else weights(std::false_type{});
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
#pragma unroll
          for (int w = 0; w < kVWords; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const unsigned sel = half == 0 ? 0x5410u : 0x7632u;
              const uint32_t x0 = __byte_perm(v[0][w], v[1][w], sel), x1 = __byte_perm(v[2][w], v[3][w], sel);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t a0 = v_pair(x0, 2 * k), a1 = v_pair(x0, 2 * k + 1);
                const uint32_t a2 = v_pair(x1, 2 * k), a3 = v_pair(x1, 2 * k + 1);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma_bf16(o[n][w * 4 + half * 2 + k], a0, a1, a2, a3, pt[n][b][0], pt[n][b][1]);
              }
            }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (++stage_out == L::kStages) stage_out = 0;
      issue();
    }

    // the next item's copies fly while this one's results are joined
    const bool more = next_segment(segments + (which ^ 1));
    if (more) start(segments[which ^ 1]);

    // join the warps
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], sh);
        off[i] += __shfl_xor_sync(0xffffffffu, off[i], sh);
      }
      if (g == 0) ml[warp * kRows + (i / 2) * 8 + 2 * j + (i & 1)] = make_float2(m[i], l[i]);
    }
    // a CTA is the first piece of one item that goes on, and a later piece of one, at most
    const int slot = 2 * blockIdx.x + (static_cast<int>(blockIdx.x) == q.first ? 1 : 0);
    float* part = partial + static_cast<int64_t>(slot) * kRows * (D + 2);
#pragma unroll
    for (int pass = 0; pass < kRows / L::kPass; ++pass) {
      __syncthreads();  // ml is written; the last pass's readers are done
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * 8 / L::kPass != pass) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* dst = join + (warp * L::kPass + n * 8 % L::kPass + 2 * j + e) * L::kPitch + g * L::kGroup;
#pragma unroll
          for (int u = 0; u < D / 16; ++u)
            *reinterpret_cast<float2*>(dst + 2 * u) =
                make_float2(fmaf(64.0f, o[n][u][e], off[2 * n + e]), fmaf(4.0f, o[n][u][2 + e], off[2 * n + e]));
        }
      }
      __syncthreads();
      // four elements a thread
      for (int i = threadIdx.x; i < L::kPass * (D / 4); i += kWarps * 32) {
        const int pr = i / (D / 4), d = i % (D / 4) * 4;
        const int rr = pass * L::kPass + pr;
        if (rr >= rows) break;
        float top = -FLT_MAX;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * kRows + rr].x);
        float sum = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 t = ml[w * kRows + rr];
          const float k = ex2(t.x - top);
          sum = fmaf(k, t.y, sum);
          const float* src = join + (w * L::kPass + pr) * L::kPitch + d + 2 * (d / (D / 8));
          const float2 u0 = *reinterpret_cast<const float2*>(src), u1 = *reinterpret_cast<const float2*>(src + 2);
          v.x = fmaf(k, u0.x, v.x); v.y = fmaf(k, u0.y, v.y); v.z = fmaf(k, u1.x, v.z); v.w = fmaf(k, u1.y, v.w);
        }
        if (q.pieces == 1) {
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          *reinterpret_cast<uint2*>(a.out + row_out[rr] + d) = make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
        } else {
          *reinterpret_cast<float4*>(part + rr * D + d) = v;
          if (d == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * rr) = make_float2(top, sum);
        }
      }
    }
    if (q.pieces > 1) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) *last_flag = atomicAdd(counters + q.first, 1u) == static_cast<unsigned>(q.pieces - 1);
      __syncthreads();
      if (*last_flag) {
        __threadfence();
        if (threadIdx.x == 0) counters[q.first] = 0;
        // a thread's elements lie in one row: its maximum first, then the sums
        constexpr int kLanes = kWarps * 32 / kRows;  // threads of a row
        const int rr = threadIdx.x / kLanes, lane_in_row = threadIdx.x % kLanes;
        constexpr int64_t kSlot = kRows * (D + 2);
        // piece 0 in slot 1 of its CTA, the others in slot 0 of theirs
        auto piece = [&](int k) { return partial + (2 * static_cast<int64_t>(q.first + k) + (k == 0 ? 1 : 0)) * kSlot; };
        if (rr < rows) {
          float top = -FLT_MAX;
          for (int k = lane_in_row; k < q.pieces; k += kLanes)
            top = fmaxf(top, __ldcg(piece(k) + kRows * D + 2 * rr));
          if constexpr (kLanes > 1) {
            const unsigned peers = (kLanes < 32 ? (1u << (kLanes & 31)) - 1u : 0xffffffffu) << (lane / kLanes * kLanes);
#pragma unroll
            for (int x2 = kLanes / 2; x2 > 0; x2 >>= 1) top = fmaxf(top, __shfl_xor_sync(peers, top, x2));
          }
          constexpr int kVecs = D / 4 / kLanes;  // float4 of a thread
          constexpr int kAtOnce = kVecs < 4 ? kVecs : 4;
          for (int v0 = 0; v0 < kVecs; v0 += kAtOnce) {
            float4 v[kAtOnce];
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll(16 / kAtOnce)
            for (int k = 0; k < q.pieces; ++k) {
              const float* src = piece(k);
              const float2 t = __ldcg(reinterpret_cast<const float2*>(src + kRows * D + 2 * rr));
              const float w = ex2(t.x - top);
              sum = fmaf(w, t.y, sum);
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) {
                const float4 u = __ldcg(reinterpret_cast<const float4*>(src + rr * D) + (v0 + i) * kLanes + lane_in_row);
                v[i].x = fmaf(w, u.x, v[i].x); v[i].y = fmaf(w, u.y, v[i].y);
                v[i].z = fmaf(w, u.z, v[i].z); v[i].w = fmaf(w, u.w, v[i].w);
              }
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
              *reinterpret_cast<uint2*>(a.out + row_out[rr] + ((v0 + i) * kLanes + lane_in_row) * 4) =
                  make_uint2(pack2(v[i].x * inv, v[i].y * inv), pack2(v[i].z * inv, v[i].w * inv));
          }
        }
      }
    }
    __syncthreads();  // the buffers are free for the next item
    if (!more) break;
  }
  // never leave with a copy in flight
  for (int s = 0; s < L::kStages; ++s)
    if ((armed >> s) & 1u) mbar_wait(bar0 + 8 * s, (phases >> s) & 1u, nullptr);
}

constexpr int kMaxCtas = 4;  // per SM, of any variant

size_t counter_bytes() { return (size_t(num_sms()) * kMaxCtas * 4 + 255) / 256 * 256; }

template <int D, int NT>
size_t partial_bytes() {
  return size_t(num_sms()) * Split<D, NT>::kCtas * 2 * Split<D, NT>::kRows * (D + 2) * 4;
}

// Counters, then two partial results a CTA of the variant that needs most.
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
  return launch_kernel(kernel, dim3(num_sms() * L::kCtas), dim3(kWarps * 32), L::kSmem, stream, 1, a, c,
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
  // the rows of a request and kv head, at most
  const int64_t tokens = max_query_len > 0 && max_query_len < num_tokens ? max_query_len : num_tokens;
  const int64_t rows = tokens * (num_heads / num_kv_heads);
  unsigned* counters = static_cast<unsigned*>(workspace);
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + counter_bytes());
  cudaError_t err;
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
