// ple_proj_mx8 and ple_gated_mx8: products of 8-bit tensors (mx8.cuh) on the
// 5th-generation tensor cores, which take the blocks' scales with the codes.
//
//   ple_proj_mx8    out = residual + x W^T, rounded once to bf16
//   ple_gated_mx8   h = act(x Wg^T) * (x Wu^T), quantised as it is computed
//
// Two kernels. For many tokens a pair of CTAs takes 256 tokens against 256
// rows of W: bound by the tensor cores, their operands' way into the SMs and
// the power limit. 8192 tokens, 16384 -> 4096: 316 to 337 us (3.3 to 3.5 PFLOP/s)
// in short runs, 380 in long ones, where the clock falls to 1.7 GHz; gated, 4096
// -> 16384: 686 to 701 us (3.2). For few tokens a CTA takes 128 rows of W against all of
// them, its columns shared out in a cluster: bound by reading W and some 4.5 us
// of start and end. One token, gated 4096 -> 16384: 24.5 to 24.9 us (5.6 TB/s),
// 16384 -> 4096: 14.5 to 15.1 (4.7); 203 tokens: 22.5 to 23.1.
#include "mx8_rule.h"
#include "mx8_tensor.cuh"

#include <algorithm>
#include <atomic>

namespace ple {
namespace {

struct ProductArgs {
  const uint8_t *x, *x_scales, *w, *w_scales;
  int64_t T;
  int E, N;  // columns; rows of the result: of W, or half as many
  int gelu;
  int wide;  // rows of out and the residual may be taken 8 bytes at a time
  const ple_bf16_t* residual;
  int64_t residual_stride;
  ple_bf16_t* out;
  uint8_t *codes, *scales;
};

// g / (1 + exp(-t)) with t = g, or gelu's 2 sqrt(2 / pi) (g + 0.044715 g^3). The
// exponential is of -|t|: nothing overflows, and gates far below keep their
// value down to float32's least exponential. Its argument is not rounded to
// fewer bits and the reciprocal, of a sum in [1, 2], is off by 2^-23 at most,
// so all of it stays below 2^-21 of the result (gelu: and 5 |t| 2^-24 of it,
// the roundings of t). The fast exponential is off by 2^-17 at t = -80 and
// moved codes that float32 does not, and the fast quotient by 1 + exp(-t) gave
// zeros from t = -87 on, a gelu's gate of -10. What it costs: 8192 tokens,
// 4096 -> 16384, 688 us against 677 with them, 777 tokens 27.2 against 26.4.
__device__ __forceinline__ float activation(float g, int gelu) {
  const float t = gelu ? g * fmaf(0.07135481282553f * g, g, 1.5957691216057308f) : g;
  const float e = expf(-fabsf(t));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * ((t >= 0.0f ? 1.0f : e) * r);
}

// ---------------------------------------------------------------------------
// Many tokens: a pair of CTAs, 256 tokens x 256 rows of W
// ---------------------------------------------------------------------------
// Each CTA stages its own 128 tokens and half of the tile's W rows (gated:
// one the gate's 128 rows, the other the 128 rows of the other half that meet
// them, so that a thread of the epilogue finds both in its row), and the
// scales of its tokens and of all W rows. A stage holds 256 columns; its
// scales go to tensor memory in front of its products, by copies of the
// products' own queue. (Brought by other warps through registers they came
// too late: 556 us against 375 for 8192 tokens, 16384 -> 4096, then.)
// One lane of a warp that stays converged issues: the operands are uniform
// registers then, and the copies cost nothing beside the products. (Issued
// under a branch on the lane, each instruction took some 70 cycles, and a
// stage 1418 instead of its products' 1024.)
// The sums take 256 of the 512 columns of tensor memory and the scales 72, so
// there is one set of sums: the epilogue's eight warps take them out, some
// 2000 cycles a tile, and give the place back before they store anything. (A
// second set that shares 72 columns with the first was no faster with tiles of
// 32 and 64 atoms, where what counts between two tiles is when their operands
// arrive; with 16 it was not tried.)
// Tiles are walked in groups of 4096 tokens, tokens first: W is read once for
// each group, and the group's tokens stay in L2. (Groups of 2048, 1024: gated
// 8192 tokens 680, 710 us against 657, all three with a shorter activation.)
//
// Warps: 0 copies, 1 issues, 2-9 the epilogue: two for each quarter of the
// rows, half of the columns each.
constexpr int kPairStages = 3;
constexpr int kPairAtoms = 2;                              // 128 columns each, of a stage
constexpr int kAtom = 128 * 128;                           // bytes of 128 rows' codes of 128 columns
constexpr int kPairScales = kPairAtoms * 3 * kMxPiece;     // bytes of a stage's scales: x, two of W
constexpr int kPairStage = kPairAtoms * 2 * kAtom + kPairScales;
constexpr int kAtScales = kPairStages * kPairAtoms * 2 * kAtom;
constexpr int kAtRoom = kAtScales + kPairStages * kPairScales;
constexpr int kRoomPitch = 17;                             // words of a row of the epilogue's room
constexpr int kRoom = 32 * kRoomPitch * 4;                 // bytes of it for a warp
constexpr int kPairEpilogue = 8;                           // warps
constexpr int kAtBars = kAtRoom + kPairEpilogue * kRoom;
constexpr int kPairBars = 2 * kPairStages + 3;
constexpr int kPairSmem = kAtBars + (kPairBars + 1) * 8 + 16 + 1024;  // and alignment
constexpr int kPairThreads = 64 + 32 * kPairEpilogue;
constexpr int kGroupTiles = 16;                            // of 256 tokens
constexpr int kScaleCols = 256;                            // scales stand behind the sums
constexpr int kAtomCols = 12;                              // 4 of x, 8 of W
static_assert(kScaleCols + kPairStages * kPairAtoms * kAtomCols <= 512, "tensor memory");
static_assert(kPairSmem <= 227 << 10, "shared memory");

// A place in a ring of buffers, the parity of its round, and which copies
// were last asked for.
template <int kPlaces>
struct Ring {
  int at = 0;
  uint32_t phase = 0, armed = 0, armed_parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == kPlaces) { at = 0; phase ^= 1u; }
  }
  __device__ __forceinline__ void arm() {
    armed |= 1u << at;
    armed_parity = (armed_parity & ~(1u << at)) | phase << at;
  }
};

struct PairTile {
  int m, n;  // first token; first row of the result
};

__device__ __forceinline__ PairTile pair_tile(int u, int m_tiles, int n_tiles, int rows) {
  const int group = u / (kGroupTiles * n_tiles), first = group * kGroupTiles;
  const int height = min(m_tiles - first, kGroupTiles), r = u - first * n_tiles;
  return {(first + r % height) * 256, r / height * rows};
}

// ---- 32 columns of bf16 rows at any address, between memory and threads ----
// A thread has a row, memory is read and written by words of two elements,
// 16 lanes a row. Word w of a row holds elements 2w and 2w + 1, or 2w - 1 and
// 2w where the row begins at an odd place: every word lies on 4 bytes, and
// only a row's ends are single elements. Rows an even number apart begin
// alike, so a lane's place in its rows never changes.

// 1 if row `row` begins at an odd place.
__device__ __forceinline__ int odd_place(const ple_bf16_t* first, int64_t stride, int row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(first) >> 1) + (row & stride)) & 1;
}

// What a lane takes of its rows' words: both elements, or one of them at a
// row's ends. Decided once for all rows, so that nothing waits between them.
struct RowPlace {
  int64_t at;  // from the first row's first element
  bool low, high;
  __device__ __forceinline__ RowPlace(const ple_bf16_t* first, int64_t stride, int columns, int lane) {
    const int e = 2 * (lane % 16) - odd_place(first, stride, lane / 16);
    at = lane / 16 * stride + e;
    low = e >= 0 && e < columns;
    high = e + 1 < columns;
  }
};

struct RowWords {
  uint32_t words[16];  // of rows 2i and 2i + 1, a half warp each
  uint32_t last;       // this lane's row's word 16, if it begins at an odd place
  bool upper;          // words hold an upper element alone
  __device__ __forceinline__ void ask(const ple_bf16_t* first, int64_t stride, int rows, int columns, int lane) {
    const RowPlace p(first, stride, columns, lane);
    const ple_bf16_t* at = first + p.at + (p.low ? 0 : 1);
    const int mine = rows - lane / 16;
    upper = !p.low;
#pragma unroll
    for (int i = 0; i < 16; ++i) words[i] = 0;
    last = 0;
    if (p.low && p.high) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (2 * i < mine) words[i] = *reinterpret_cast<const uint32_t*>(at + 2 * i * stride);
    } else if (p.low || p.high) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (2 * i < mine) words[i] = at[2 * i * stride];
    }
    if (lane < rows && columns == 32 && odd_place(first, stride, lane)) last = first[lane * stride + 31];
  }
  __device__ __forceinline__ void stage(uint32_t* room, int lane) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) room[(2 * i + lane / 16) * kRoomPitch + lane % 16] = upper ? words[i] << 16 : words[i];
    room[lane * kRoomPitch + 16] = last;
  }
};

// This thread's row out of the room, as pairs of elements, and into it.
__device__ __forceinline__ void take_row(uint32_t (&pairs)[16], const uint32_t* row, int odd) {
  uint32_t w = row[0];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t next = row[i + 1];
    pairs[i] = odd ? __byte_perm(w, next, 0x5432) : w;
    w = next;
  }
}
__device__ __forceinline__ void put_row(const uint32_t (&pairs)[16], uint32_t* row, int odd) {
  uint32_t before = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    row[i] = odd ? __byte_perm(before, pairs[i], 0x5432) : pairs[i];
    before = pairs[i];
  }
  row[16] = before >> 16;
}

__device__ __forceinline__ void store_rows(const uint32_t* room, ple_bf16_t* first, int64_t stride, int rows, int columns, int lane) {
  const RowPlace p(first, stride, columns, lane);
  ple_bf16_t* const at = first + p.at;
  const int mine = rows - lane / 16;
  uint32_t words[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) words[i] = room[(2 * i + lane / 16) * kRoomPitch + lane % 16];
  const uint32_t last = room[lane * kRoomPitch + 16];
  if (p.low && p.high) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (2 * i < mine) *reinterpret_cast<uint32_t*>(at + 2 * i * stride) = words[i];
  } else if (p.low) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (2 * i < mine) at[2 * i * stride] = static_cast<ple_bf16_t>(words[i]);
  } else if (p.high) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (2 * i < mine) at[2 * i * stride + 1] = static_cast<ple_bf16_t>(words[i] >> 16);
  }
  if (lane < rows && columns == 32 && odd_place(first, stride, lane)) first[lane * stride + 31] = static_cast<ple_bf16_t>(last);
}

template <bool kGated>
__global__ void __launch_bounds__(kPairThreads, 1)
product_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_xs, const __grid_constant__ CUtensorMap map_ws,
                    const ProductArgs a, int32_t* dev_err) {
  constexpr int kRows = kGated ? 128 : 256;  // of the result in a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem), bar0 = base + kAtBars;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto free = [&](int s) { return bar0 + 8u * (kPairStages + s); };
  const uint32_t sums_full = bar0 + 8u * (2 * kPairStages), sums_free = sums_full + 8, done = sums_full + 16;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + kAtBars + kPairBars * 8);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* const kind = abort_flag + 1;  // of activation
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const int m_tiles = static_cast<int>((a.T + 255) / 256), n_tiles = (a.N + kRows - 1) / kRows;
  const int units = m_tiles * n_tiles;
  const int atoms = a.E / 128, stages = (atoms + kPairAtoms - 1) / kPairAtoms;
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(full(s), 1);  // the even CTA's expect_tx; bytes of both
      mbar_init(free(s), 1);
    }
    mbar_init(sums_full, 1);
    mbar_init(sums_free, 2 * kPairEpilogue);
    mbar_init(done, 1);
    mbar_fence_init();
    *abort_flag = 0;
    *kind = a.gelu;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  cluster_barrier();  // both CTAs' barriers and tensor memory are there
  fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 0 && lane == 0) {
    // ---------------- copies (both CTAs) ----------------
    prefetch_map(&map_x);
    prefetch_map(&map_w);
    prefetch_map(&map_xs);
    prefetch_map(&map_ws);
    int s = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true;
    for (int u = pair; ok && u < units; u += pairs) {
      const PairTile t = pair_tile(u, m_tiles, n_tiles, kRows);
      const int m = t.m + static_cast<int>(rank) * 128;
      const int n = kGated ? static_cast<int>(rank) * a.N + t.n : t.n + static_cast<int>(rank) * 128;  // this CTA's W rows
      const int piece[3] = {m / 128 * atoms, t.n / 128 * atoms, (kGated ? a.N + t.n : t.n + 128) / 128 * atoms};  // scales: of all W rows
      for (int k = 0; k < stages; ++k) {
        if (!mbar_wait(free(s), phase ^ 1u, abort_flag)) { ok = false; break; }
        const uint32_t bar = at_rank(full(s), 0);
        if (rank == 0) {
          mbar_arrive_expect_tx(full(s), 2 * kPairStage);
          armed |= 1u << s;
          armed_parity = (armed_parity & ~(1u << s)) | (phase << s);
        }
        // past the last column (an odd number of atoms) zeros come
        tma_load_pair(base + s * 2 * kPairAtoms * kAtom, &map_x, bar, k * kPairAtoms, m);
        tma_load_pair(base + (s * 2 + 1) * kPairAtoms * kAtom, &map_w, bar, k * kPairAtoms, n);
        const uint32_t to = base + kAtScales + s * kPairScales;
        tma_load_2d_pair(to, &map_xs, bar, 0, piece[0] + k * kPairAtoms);
        for (int h = 0; h < 2; ++h)
          tma_load_2d_pair(to + (1 + h) * kPairAtoms * kMxPiece, &map_ws, bar, 0, piece[1 + h] + k * kPairAtoms);
        if (++s == kPairStages) { s = 0; phase ^= 1u; }
      }
    }
    if (!ok) { *abort_flag = 1; set_dev_err(dev_err, PLE_DEVERR_TIMEOUT); }
    // no leaving with copies in flight
    for (int i = 0; i < kPairStages; ++i)
      if (armed & (1u << i)) mbar_wait(full(i), (armed_parity >> i) & 1u, nullptr);
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------- products (the even CTA, for both) ----------------
      // The whole warp goes through the loop and one lane issues: operands
      // are uniform registers then.
      const uint32_t sums = __shfl_sync(0xffffffffu, tmem, 0);
      int s = 0;
      uint32_t phase = 0, tile_phase = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += pairs, tile_phase ^= 1u) {
        if (!(ok = __all_sync(0xffffffffu, wait_for(sums_free, tile_phase ^ 1u, abort_flag)))) break;
        fence_after();
        for (int k = 0; k < stages; ++k) {
          if (!(ok = __all_sync(0xffffffffu, wait_for(full(s), phase, abort_flag)))) break;
          fence_after();
          if (elected()) {
#pragma unroll
            for (int i = 0; i < kPairAtoms; ++i)
#pragma unroll
              for (int j = 0; j < 3; ++j)
                scales_to_tmem<2>(sums + kScaleCols + (s * kPairAtoms + i) * kAtomCols + 4 * j,
                                  base + kAtScales + s * kPairScales + (j * kPairAtoms + i) * kMxPiece);
#pragma unroll
            for (int i = 0; i < kPairAtoms; ++i) {
              if (k * kPairAtoms + i >= atoms) break;  // its scales are another row's
              const uint32_t scales = sums + kScaleCols + (s * kPairAtoms + i) * kAtomCols;
              const uint64_t x = codes_operand(base + (s * 2 * kPairAtoms + i) * kAtom);
              const uint64_t w = codes_operand(base + ((s * 2 + 1) * kPairAtoms + i) * kAtom);
#pragma unroll
              for (int b = 0; b < 4; ++b)
                mma_mx8<2>(sums, x + 2 * b, w + 2 * b, mx_idesc(256, 256) | mx_block(b), scales, scales + 4, (k | i | b) != 0);
            }
            mma_commit_pair(free(s));
            if (k == stages - 1) mma_commit_pair(sums_full);
          }
          __syncwarp();
          if (++s == kPairStages) { s = 0; phase ^= 1u; }
        }
      }
      if (!ok && lane == 0) { *abort_flag = 1; set_dev_err(dev_err, PLE_DEVERR_TIMEOUT); }
      __syncwarp();
      // however the loop ended, no product reads or writes after this
      if (elected())
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(done) : "memory");
      __syncwarp();
      if (!wait_for(done, 0, nullptr) && lane == 0) { *abort_flag = 1; set_dev_err(dev_err, PLE_DEVERR_TIMEOUT); }
    }
    __syncwarp();
  } else if (warp >= 2) {
    // ---------------- epilogue (both CTAs) ----------------
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint32_t tile_phase = 0;
    for (int u = pair; u < units; u += pairs, tile_phase ^= 1u) {
      const PairTile t = pair_tile(u, m_tiles, n_tiles, kRows);
      const int64_t m0 = t.m + static_cast<int64_t>(rank) * 128 + quad * 32;
      const int rows = static_cast<int>(min(max(a.T - m0, int64_t(0)), int64_t(32)));  // of this warp's that exist
      // The residual is brought while the products run, all of it: beside
      // their operands a load takes some 3000 cycles.
      uint32_t pairs[kGated ? 1 : 4][16];
      uint32_t* const room = reinterpret_cast<uint32_t*>(smem + kAtRoom) + (warp - 2) * 32 * kRoomPitch;
      if constexpr (!kGated) {
        if (a.residual != nullptr) {
          const ple_bf16_t* const first = a.residual + m0 * a.residual_stride + t.n + half * 128;
          RowWords words[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) words[c].ask(first + 32 * c, a.residual_stride, rows, min(32, a.N - t.n - half * 128 - 32 * c), lane);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            words[c].stage(room, lane);
            __syncwarp();
            take_row(pairs[c], room + lane * kRoomPitch, odd_place(first, a.residual_stride, lane));
            __syncwarp();
          }
        }
      }
      if (!__all_sync(0xffffffffu, sums_wait(sums_full, tile_phase, abort_flag, stages))) {
        if (lane == 0) { *abort_flag = 1; set_dev_err(dev_err, PLE_DEVERR_TIMEOUT); }
        break;
      }
      fence_after();
      auto release = [&]() {
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(at_rank(sums_free, 0));
      };
      if constexpr (kGated) {
        // 64 columns of the gate and the 64 that meet them
        float v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ask(lanes + c / 2 * 128 + half * 64 + c % 2 * 32, v[c]);
        tmem_wait(v);
        release();
        // read only now, so that no part of the activations comes in front of
        // the release (8192 tokens, 4096 -> 16384: 688 us, 725 with a.gelu)
        const int gelu = *kind;
        const int64_t m = m0 + lane;
        uint32_t word = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[c][i] = activation(v[c][i], gelu) * v[c + 2][i];
            top = max(top, abs_bits(v[c][i]));
          }
          const uint32_t b = mx_scale_byte(top);
          const float by = mx_inverse(b);
          word |= b << (8 * c);
          uint32_t codes[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            codes[i] = mx_codes4(v[c][4 * i] * by, v[c][4 * i + 1] * by, v[c][4 * i + 2] * by, v[c][4 * i + 3] * by);
          if (m < a.T) store32(a.codes + m * a.N + t.n + half * 64 + c * 32, codes);
        }
        if (m < a.T) *reinterpret_cast<uint16_t*>(a.scales + mx_scale_at(m, (t.n + half * 64) / 32, a.N)) = static_cast<uint16_t>(word);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float y[32];
          tmem_load(lanes + half * 128 + c * 32, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (a.residual != nullptr) {
              y[2 * i] += bf_lo(pairs[c][i]);
              y[2 * i + 1] += bf_hi(pairs[c][i]);
            }
            pairs[c][i] = pack2(y[2 * i], y[2 * i + 1]);
          }
        }
        release();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = t.n + half * 128 + c * 32;
          if (n >= a.N) break;
          ple_bf16_t* const first = a.out + m0 * a.N + n;
          put_row(pairs[c], room + lane * kRoomPitch, odd_place(first, a.N, lane));
          __syncwarp();
          store_rows(room, first, a.N, rows, min(32, a.N - n), lane);
          __syncwarp();
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  cluster_barrier();  // no CTA leaves while the other's products read its memory
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Pairs of CTAs that can be on the GPU at once (a GPC may not hold a whole
// number of pairs), of a kernel on the current device.
template <bool kGated>
int resident_pairs() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev >= 0 && dev < kDevices && known[dev].load() > 0) return known[dev].load();
  int pairs = num_sms() / 2, active = 0;
  cudaFuncSetAttribute(product_pair_kernel<kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);  // else none fits
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs) * 2);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&active, product_pair_kernel<kGated>, &cfg) == cudaSuccess && active > 0)
    pairs = active < pairs ? active : pairs;
  else
    cudaGetLastError();  // a failed query leaves the SMs' bound
  if (dev >= 0 && dev < kDevices) known[dev].store(pairs);
  return pairs;
}

template <bool kGated>
ple_status launch_pair(const ProductArgs& a, int32_t* dev_err, cudaStream_t stream, const char* name) {
  const int64_t w_rows = kGated ? 2 * int64_t(a.N) : a.N;
  CUtensorMap x, w, xs, ws;
  ple_status s = mx_codes_map(&x, a.x, a.T, a.E, 128, kPairAtoms, name);
  if (s == PLE_OK) s = mx_codes_map(&w, a.w, w_rows, a.E, 128, kPairAtoms, name);
  if (s == PLE_OK) s = mx_scales_map(&xs, a.x_scales, a.T, a.E, kPairAtoms, name);
  if (s == PLE_OK) s = mx_scales_map(&ws, a.w_scales, w_rows, a.E, kPairAtoms, name);
  if (s != PLE_OK) return s;
  const auto kernel = product_pair_kernel<kGated>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (err != cudaSuccess) return check_cuda(err, name);
  const int64_t units = (a.T + 255) / 256 * ((a.N + (kGated ? 127 : 255)) / (kGated ? 128 : 256));
  if (units > INT32_MAX / 2) return fail(PLE_ERR_UNSUPPORTED, "%s: %lld tokens", name, static_cast<long long>(a.T));
  const int64_t pairs = std::min<int64_t>(units, resident_pairs<kGated>());
  return check_cuda(launch_kernel(kernel, dim3(static_cast<unsigned>(2 * pairs)), dim3(kPairThreads), kPairSmem, stream, 2,
                                  x, w, xs, ws, a, dev_err), name);
}

// ---------------------------------------------------------------------------
// Few tokens: a CTA takes 128 rows of W
// ---------------------------------------------------------------------------
// W is the first operand (128 rows fill the tensor cores' lanes), the tokens
// the second: 16 to 256 of them. Gated, a CTA takes 128 rows of the gate and
// the 128 that meet them, into sums of their own. Where the rows alone would
// leave SMs without work, a cluster of CTAs shares them: each takes a part of
// the columns, and their sums meet through distributed shared memory, in the
// order of the CTAs, each joining (and finishing) a share of the tokens.
// Up to 64 tokens two CTAs share an SM: more of them are ready to ask for W
// than SMs are there, and one starts while another ends (16384 -> 4096, 64
// tokens: 18.4 us against 21.2 with one). A stage is one atom of columns: two
// would leave too few of them (one token, 16384 -> 4096: 17.8 us against 15.7).
// W's first stages are asked into L2 while the kernel before still runs, which
// reads nothing of them and so may not wait for it (15.7 -> 14.8 with the
// rest of the start).
//
// Warps: 0 copies, 1 issues, 2-5 take the sums out; all eight join.
constexpr int kFewThreads = 256;

template <bool kGated, int kTokens>
struct Few {
  static constexpr int kSides = kGated ? 2 : 1;  // of W
  static constexpr int kXPieces = kTokens > 128 ? 2 : 1;
  static constexpr int kResident = few_resident(kTokens);        // CTAs an SM
  static constexpr int kMaxParts = few_max_parts(kTokens);       // CTAs that share the columns
  static constexpr int kCodes = kSides * kAtom + kTokens * 128;  // bytes of a stage: an atom
  static constexpr int kScales = (kSides + kXPieces) * kMxPiece;
  static constexpr int kBudget = kResident == 2 ? 110 << 10 : 220 << 10;
  static constexpr int kFit = kBudget / (kCodes + kScales);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kAtScales = kStages * kCodes;
  static constexpr int kAtBars = kAtScales + kStages * kScales;
  static constexpr int kSmem = kAtBars + (2 * kStages + 2) * 8 + 16 + 1024;  // and alignment
  static constexpr int kAsk = kTokens < 32 ? 16 : 32;            // tokens a thread takes out at once
  static constexpr int kBatch = 16 / (kMaxParts * kSides);       // tokens a warp joins at once
  static constexpr int kCols = kSides * kTokens;                 // of sums
  static constexpr int kStageCols = 4 * (kSides + kXPieces);     // of scales
  static constexpr int kNeed = kCols + kStages * kStageCols;
  static constexpr int kTmem = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  static_assert(kNeed <= 512 / kResident && kTmem <= 512 / kResident, "tensor memory");
  static_assert(kTokens * kSides * 128 * 4 <= kAtScales, "the sums fit where the codes were");
  static_assert(kStages >= 2, "stages");
};

template <bool kGated, int kTokens>
__global__ void __launch_bounds__(kFewThreads, Few<kGated, kTokens>::kResident)
product_few_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                   const ProductArgs a, int parts, int wide, int32_t* dev_err) {
  using L = Few<kGated, kTokens>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem), bar0 = base + L::kAtBars;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto free = [&](int s) { return bar0 + 8u * (L::kStages + s); };
  const uint32_t sums_full = bar0 + 8u * (2 * L::kStages);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kAtBars + (2 * L::kStages + 2) * 8);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int part = blockIdx.x % parts, n0 = blockIdx.x / parts * 128;
  const int64_t t0 = int64_t(blockIdx.y) * kTokens;
  const int tokens = static_cast<int>(min(a.T - t0, int64_t(kTokens)));
  const int atoms = a.E / 128;
  const int first = static_cast<int>(int64_t(part) * atoms / parts), last = static_cast<int>(int64_t(part + 1) * atoms / parts);

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(free(s), 1);
    }
    mbar_init(sums_full, 1);
    mbar_fence_init();
    *abort_flag = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(L::kTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp == 0 && lane == 0) {
    // W into L2 while the kernel before this one ends: nothing is read of it
    prefetch_map(&map_w);
    prefetch_map(&map_x);
    for (int k = first; k < last && k < first + L::kStages; ++k)
      for (int i = 0; i < L::kSides; ++i) prefetch_atoms(&map_w, k, i * a.N + n0);
  }
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- copies ----------------
      Ring<L::kStages> ring;
      bool ok = true;
      const uint8_t* const xs = a.x_scales + t0 / 128 * atoms * kMxPiece;  // (t0 is 0, or blocks are of 128 or 256)
      const uint8_t* ws[2];
      for (int i = 0; i < L::kSides; ++i) ws[i] = a.w_scales + (int64_t(i) * a.N + n0) / 128 * atoms * kMxPiece;
      // the second 128 tokens' scales, where there are such tokens
      const bool more = L::kXPieces == 2 && tokens > 128;
      for (int k = first; k < last; ++k, ring.next()) {
        const int s = ring.at;
        if (!(ok = mbar_wait(free(s), ring.phase ^ 1u, abort_flag))) break;
        mbar_arrive_expect_tx(full(s), L::kSides * kAtom + wide * 128 + kMxPiece * (L::kSides + (more ? 2 : 1)));
        ring.arm();
        const uint32_t to = base + s * L::kCodes, scales = base + L::kAtScales + s * L::kScales;
        for (int i = 0; i < L::kSides; ++i) {
          tma_load_atoms(to + i * kAtom, &map_w, full(s), k, i * a.N + n0);
          bulk_copy_g2s(scales + i * kMxPiece, ws[i] + int64_t(k) * kMxPiece, kMxPiece, full(s));
        }
        tma_load_atoms(to + L::kSides * kAtom, &map_x, full(s), k, static_cast<int>(t0));
        bulk_copy_g2s(scales + L::kSides * kMxPiece, xs + int64_t(k) * kMxPiece, kMxPiece, full(s));
        if (more)
          bulk_copy_g2s(scales + (L::kSides + 1) * kMxPiece, xs + int64_t(atoms + k) * kMxPiece, kMxPiece, full(s));
      }
      if (!ok) { *abort_flag = 1; set_dev_err(dev_err, PLE_DEVERR_TIMEOUT); }
      for (int i = 0; i < L::kStages; ++i)
        if (ring.armed >> i & 1u) mbar_wait(full(i), ring.armed_parity >> i & 1u, nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- products: one lane issues, in code that the whole warp runs ----------------
    const uint32_t sums = __shfl_sync(0xffffffffu, tmem, 0);
    Ring<L::kStages> ring;
    bool ok = true;
    for (int k = first; k < last; ++k, ring.next()) {
      const int s = ring.at;
      if (!(ok = __all_sync(0xffffffffu, wait_for(full(s), ring.phase, abort_flag)))) break;
      fence_after();
      if (elected()) {
        const uint32_t from = base + L::kAtScales + s * L::kScales, scales = sums + L::kCols + s * L::kStageCols;
#pragma unroll
        for (int i = 0; i < L::kSides + L::kXPieces; ++i) scales_to_tmem<1>(scales + 4 * i, from + i * kMxPiece);
        const uint64_t x = codes_operand(base + s * L::kCodes + L::kSides * kAtom);
#pragma unroll
        for (int i = 0; i < L::kSides; ++i) {
          const uint64_t w = codes_operand(base + s * L::kCodes + i * kAtom);
#pragma unroll
          for (int b = 0; b < 4; ++b)
            mma_mx8<1>(sums + i * kTokens, w + 2 * b, x + 2 * b, mx_idesc(128, wide) | mx_block(b), scales + 4 * i,
                       scales + 4 * L::kSides, k > first || b > 0);
        }
        mma_commit(free(s));
      }
      __syncwarp();
    }
    // Before the commit: the sums' warps see that these are none.
    if (!ok && lane == 0) { *abort_flag = 1; set_dev_err(dev_err, PLE_DEVERR_TIMEOUT); }
    __syncwarp();
    // however the loop ended, no product reads or writes after this
    if (elected()) mma_commit(sums_full);
    __syncwarp();
    if (!wait_for(sums_full, 0, nullptr) && lane == 0) { *abort_flag = 1; set_dev_err(dev_err, PLE_DEVERR_TIMEOUT); }
  } else if (warp < 6) {
    // ---------------- sums, where the codes were: [token][side][row] ----------------
    const bool ok = __all_sync(0xffffffffu, sums_wait(sums_full, 0, abort_flag, last - first) && *abort_flag == 0);
    if (!ok && lane == 0) { *abort_flag = 1; set_dev_err(dev_err, PLE_DEVERR_TIMEOUT); }
    fence_after();
    if (ok) {
      const int row = (warp & 3) * 32 + lane;
      const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      float* const mine = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int i = 0; i < L::kSides; ++i)
#pragma unroll 1
        for (int c = 0; c < tokens; c += L::kAsk) {
          float v[L::kAsk];
          if constexpr (L::kAsk == 16) tmem_load16(lanes + i * kTokens + c, v);
          else tmem_load(lanes + i * kTokens + c, v);
#pragma unroll
          for (int j = 0; j < L::kAsk; ++j)
            if (c + j < tokens) mine[((c + j) * L::kSides + i) * 128 + row] = v[j];
        }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::kTmem) : "memory");
  }
  if (parts > 1) cluster_barrier();
  // ---------------- the parts' sums, in their order: a warp takes a token, a lane 4 rows ----------------
  // (a few tokens at once: what is far away is asked for together)
  const int n = n0 + lane * 4;
  constexpr int kStride = kFewThreads / 32;
  for (int i0 = warp; part + i0 * parts < tokens; i0 += kStride * L::kBatch) {
    float4 f[L::kBatch][L::kMaxParts][L::kSides];
    uint2 more[L::kBatch];
    auto token = [&](int q) { return part + (i0 + q * kStride) * parts; };
#pragma unroll
    for (int q = 0; q < L::kBatch; ++q) {
      const int t = token(q);
      if (t >= tokens) break;
      if (!kGated && a.wide && a.residual != nullptr && n < a.N)
        more[q] = *reinterpret_cast<const uint2*>(a.residual + (t0 + t) * a.residual_stride + n);
#pragma unroll
      for (int p = 0; p < L::kMaxParts; ++p)
        if (p < parts)
#pragma unroll
          for (int i = 0; i < L::kSides; ++i) f[q][p][i] = read_cluster4(base + ((t * L::kSides + i) * 128 + lane * 4) * 4, p);
    }
#pragma unroll
    for (int q = 0; q < L::kBatch; ++q) {
      const int64_t m = t0 + token(q);
      if (token(q) >= tokens) break;
      float v[L::kSides][4] = {};
#pragma unroll
      for (int p = 0; p < L::kMaxParts; ++p)
        if (p < parts)
#pragma unroll
          for (int i = 0; i < L::kSides; ++i) {
            v[i][0] += f[q][p][i].x; v[i][1] += f[q][p][i].y; v[i][2] += f[q][p][i].z; v[i][3] += f[q][p][i].w;
          }
      if constexpr (kGated) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[0][i] = activation(v[0][i], a.gelu) * v[1][i];
          top = max(top, abs_bits(v[0][i]));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t b = mx_scale_byte(top);
        const float by = mx_inverse(b);
        *reinterpret_cast<uint32_t*>(a.codes + m * a.N + n) = mx_codes4(v[0][0] * by, v[0][1] * by, v[0][2] * by, v[0][3] * by);
        uint32_t word = b << (lane / 8 * 8);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        word |= __shfl_xor_sync(0xffffffffu, word, 16);
        if (lane == 0) *reinterpret_cast<uint32_t*>(a.scales + mx_scale_at(m, n0 / 32, a.N)) = word;
      } else if (a.wide) {
        if (n < a.N) {
          if (a.residual != nullptr) {
            v[0][0] += bf_lo(more[q].x); v[0][1] += bf_hi(more[q].x); v[0][2] += bf_lo(more[q].y); v[0][3] += bf_hi(more[q].y);
          }
          *reinterpret_cast<uint2*>(a.out + m * a.N + n) = make_uint2(pack2(v[0][0], v[0][1]), pack2(v[0][2], v[0][3]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < a.N) {
            if (a.residual != nullptr) v[0][i] += bf_lo(a.residual[m * a.residual_stride + n + i]);
            a.out[m * a.N + n + i] = static_cast<ple_bf16_t>(pack2(v[0][i], 0.0f) & 0xffffu);
          }
      }
    }
  }
  if (parts > 1) cluster_barrier();  // no CTA leaves while its sums are read
}

template <bool kGated, int kTokens>
ple_status launch_few(const ProductArgs& a, int32_t* dev_err, cudaStream_t stream, const char* name) {
  using L = Few<kGated, kTokens>;
  CUtensorMap x, w;
  // a tile's tokens, in the products' steps of 16: a tile of 256 that holds 130
  // is 144 wide (8192 x 4096, 14.4 us against 15.1)
  const int wide = static_cast<int>(std::min<int64_t>((a.T + 15) / 16 * 16, kTokens));
  ple_status s = mx_codes_map(&x, a.x, a.T, a.E, wide, 1, name);
  if (s == PLE_OK) s = mx_codes_map(&w, a.w, kGated ? 2 * int64_t(a.N) : a.N, a.E, 128, 1, name);
  if (s != PLE_OK) return s;
  const auto kernel = product_few_kernel<kGated, kTokens>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (err != cudaSuccess) return check_cuda(err, name);
  const int tiles = (a.N + 127) / 128, blocks = static_cast<int>((a.T + kTokens - 1) / kTokens);
  const int parts = few_parts(kTokens, int64_t(tiles) * blocks, a.E / 128, num_sms());
  const dim3 grid(static_cast<unsigned>(tiles * parts), static_cast<unsigned>(blocks));
  return check_cuda(launch_kernel(kernel, grid, dim3(kFewThreads), L::kSmem, stream, static_cast<unsigned>(parts), x, w, a,
                                  parts, wide, dev_err), name);
}

template <bool kGated>
ple_status launch_product(const ProductArgs& a, int32_t* dev_err, cudaStream_t stream, const char* name) {
  const int tile = product_tile({a.T, a.E, a.N, kGated}, num_sms(), [] { return resident_pairs<kGated>(); });
  if (tile == 32) return launch_few<kGated, 32>(a, dev_err, stream, name);
  if (tile == 128) return launch_few<kGated, 128>(a, dev_err, stream, name);
  if constexpr (kGated) {
    if (tile == 16) return launch_few<true, 16>(a, dev_err, stream, name);
  } else {
    if (tile == 64) return launch_few<false, 64>(a, dev_err, stream, name);
    if (tile == 256) return launch_few<false, 256>(a, dev_err, stream, name);
  }
  return launch_pair<kGated>(a, dev_err, stream, name);
}

ple_status check_product(const char* name, const uint8_t* x, const uint8_t* x_scales, int64_t num_tokens, int32_t in_dim,
                         const uint8_t* w, const uint8_t* w_scales, int32_t rows) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || in_dim < 1 || rows < 1)
    return fail(PLE_ERR_INVALID_ARG, "%s: %lld tokens, %d columns, %d rows", name, static_cast<long long>(num_tokens),
                in_dim, rows);
  if (in_dim % kMxTile != 0)
    return fail(PLE_ERR_UNSUPPORTED, "%s: %d columns (a multiple of %d)", name, in_dim, kMxTile);
  if (num_tokens == 0) return PLE_OK;
  if (rows > INT32_MAX - 255) return fail(PLE_ERR_UNSUPPORTED, "%s: %d rows", name, rows);  // tiles are counted in 32 bits
  if (num_tokens > 65535 * 64) return fail(PLE_ERR_UNSUPPORTED, "%s: %lld tokens", name, static_cast<long long>(num_tokens));
  if (x == nullptr || x_scales == nullptr || w == nullptr || w_scales == nullptr)
    return fail(PLE_ERR_INVALID_ARG, "%s: null codes or scales", name);
  if (!aligned16(x) || !aligned16(x_scales) || !aligned16(w) || !aligned16(w_scales))
    return fail(PLE_ERR_INVALID_ARG, "%s: codes and scales must be 16-byte aligned", name);
  return PLE_OK;
}

// True if [to, to + n) meets an operand of the product.
bool meets_operands(const void* to, size_t n, const ProductArgs& a, int64_t w_rows) {
  return overlaps(to, n, a.x, a.T * a.E) || overlaps(to, n, a.x_scales, mx_scale_size(a.T, a.E)) ||
         overlaps(to, n, a.w, w_rows * a.E) || overlaps(to, n, a.w_scales, mx_scale_size(w_rows, a.E));
}

}  // namespace

ple_status encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* at, int dims, const cuuint64_t* size,
                      const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle, const char* name) {
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return fail(PLE_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", name);
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = encode(map, type, dims, const_cast<void*>(at), size, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PLE_OK : fail(PLE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", name, static_cast<int>(r));
}

ple_status mx_codes_map(CUtensorMap* map, const void* codes, int64_t rows, int columns, int box_rows, int box_atoms,
                        const char* name) {
  const cuuint64_t size[3] = {128, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(columns) / 128};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(columns), 128};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_atoms)};
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, 3, size, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, name);
}

ple_status mx_scales_map(CUtensorMap* map, const void* scales, int64_t rows, int columns, int box_pieces, const char* name) {
  const cuuint64_t size[2] = {kMxPiece / 4, static_cast<cuuint64_t>(mx_scale_size(rows, columns) / kMxPiece)};
  const cuuint64_t strides[1] = {kMxPiece};
  const cuuint32_t box[2] = {kMxPiece / 4, static_cast<cuuint32_t>(box_pieces)};
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, 2, size, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE, name);
}

}  // namespace ple

using namespace ple;

PLE_EXPORT ple_status ple_gated_mx8(const uint8_t* x, const uint8_t* x_scales, int64_t num_tokens, int32_t hidden,
                                    const uint8_t* w, const uint8_t* w_scales, int32_t inner, int32_t activation,
                                    uint8_t* codes, uint8_t* scales, int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_gated_mx8";
  const ple_status s = check_product(name, x, x_scales, num_tokens, hidden, w, w_scales, inner);
  if (s != PLE_OK) return s;
  if (activation != PLE_SILU && activation != PLE_GELU)
    return fail(PLE_ERR_UNSUPPORTED, "%s: activation %d", name, activation);
  if (inner % kMxTile != 0 || inner > INT32_MAX / 2)
    return fail(PLE_ERR_UNSUPPORTED, "%s: inner %d (a multiple of %d)", name, inner, kMxTile);
  if (num_tokens == 0) return PLE_OK;
  if (codes == nullptr || scales == nullptr) return fail(PLE_ERR_INVALID_ARG, "%s: null codes or scales", name);
  if (!aligned16(codes) || !aligned16(scales))
    return fail(PLE_ERR_INVALID_ARG, "%s: codes and scales must be 16-byte aligned", name);
  const ProductArgs a{x, x_scales, w, w_scales, num_tokens, hidden, inner, activation == PLE_GELU, 0, nullptr, 0,
                      nullptr, codes, scales};
  const size_t n = static_cast<size_t>(num_tokens) * inner, m = mx_scale_size(num_tokens, inner);
  if (meets_operands(codes, n, a, 2LL * inner) || meets_operands(scales, m, a, 2LL * inner) || overlaps(codes, n, scales, m))
    return fail(PLE_ERR_INVALID_ARG, "%s: an output overlaps an operand or the other output", name);
  return launch_product<true>(a, dev_err, stream, name);
}

PLE_EXPORT ple_status ple_proj_mx8(const uint8_t* x, const uint8_t* x_scales, int64_t num_tokens, int32_t in_dim,
                                   const uint8_t* w, const uint8_t* w_scales, int32_t out_dim,
                                   const ple_bf16_t* residual, int64_t residual_stride, ple_bf16_t* out,
                                   int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_proj_mx8";
  const ple_status s = check_product(name, x, x_scales, num_tokens, in_dim, w, w_scales, out_dim);
  if (s != PLE_OK || num_tokens == 0) return s;
  if (out == nullptr) return fail(PLE_ERR_INVALID_ARG, "%s: null out", name);
  if (((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(residual)) & 1) != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: out or the residual at an odd address", name);
  const bool wide = out_dim % 4 == 0 && ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(residual)) & 7) == 0 &&
                    (residual == nullptr || residual_stride % 4 == 0);
  const ProductArgs a{x, x_scales, w, w_scales, num_tokens, in_dim, out_dim, 0, wide, residual, residual_stride, out,
                      nullptr, nullptr};
  const size_t n = static_cast<size_t>(num_tokens) * out_dim * 2;
  if (meets_operands(out, n, a, out_dim)) return fail(PLE_ERR_INVALID_ARG, "%s: out overlaps an operand", name);
  if (residual != nullptr && !(residual == out && (residual_stride == out_dim || num_tokens == 1)) &&
      rows_overlap({out, 1, 0, static_cast<int64_t>(n)}, {residual, num_tokens, residual_stride * 2, int64_t(out_dim) * 2}))
    return fail(PLE_ERR_INVALID_ARG, "%s: out overlaps the residual and is not the residual", name);
  return launch_product<false>(a, dev_err, stream, name);
}
