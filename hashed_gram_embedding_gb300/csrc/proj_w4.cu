// ple_proj_w4: out = x W^T with W in 4 bits, a scale and a zero point per
// group of columns, for steps of few tokens.
//
// Bound by reading the codes, half a byte a weight. Products on warp-wide
// matrix instructions (16 x 8 x 16, bf16, f32 sums): W is the A operand, 16
// output rows, and 8 tokens fill the other side. A weight's code never meets
// memory again: masked out of its word where it stands, a pair of codes is a
// pair of bf16 subnormals (c 2^-133, or c 2^-129 for the upper half of a
// byte), and one fused multiply-add makes (c - z) / 64 of it, exactly. The
// scale meets the float32 sum once per group, and 64 the whole sum (with the
// scale it would be infinite for scales that are not):
//   out[t][n] = 64 sum_g s_ng sum_{e in g} x_te (c_ne - z_ng) / 64.
// The contraction index may run in any order, so a lane reads codes in the
// widest pieces that lie in one group - 16, 8 or 4 bytes of a row for groups
// of 128, 64 or 32 columns, four lanes together a group of a row - and the
// x of the same columns, 16 bytes a word of codes.
//
// A CTA takes 16 output rows and all columns; its warps take blocks of 128
// columns in turn, each with the next blocks' codes in flight, and add their
// sums up in shared memory, in the warps' order. All codes of a small weight
// are thus asked for at once, by as many SMs as there are. Measured: one token,
// 2048 x 8192, 4.8 us (1.8 TB/s, a launch and two trips to memory), 4096 x
// 16384 12.1 us (2.9 TB/s); 13 tokens, 4096 x 4096, 6.6 us.
#include "codes.cuh"
#include "tensor_core.cuh"

namespace ple {
namespace {

constexpr int kColumns = 128;  // of a block

struct ProjArgs {
  const ple_bf16_t* x;
  int64_t x_stride;
  int64_t T;
  int E, N;
  const uint8_t* codes;
  const ple_bf16_t* scales;
  const uint8_t* zeros;
  ple_bf16_t* out;
};

template <int NT>
struct Proj {
  static constexpr int kWarps = 8;
  static constexpr int kDepth = 4;                 // blocks of codes in flight
  static constexpr int kRows = 16;
  static constexpr int kPitch = 8 * NT + 1;        // floats of a row's sums, padded
  static constexpr int kSmem = kWarps * kRows * kPitch * 4;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of a word as (c - z) / 64, with z64 a pair of -z / 64.
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int i, uint32_t z64) {
  return bf2_mad(code_bits(word, i), i % 2 == 0 ? 0x7F007F00u /* 2^127 */ : 0x7D007D00u /* 2^123 */, z64);
}

// Column of a lane's word w in a block: four lanes share a group's columns.
template <int kGroup>
__device__ __forceinline__ int column_of(int w, int j) {
  constexpr int kWords = kGroup / 32;  // of a lane and group
  return w / kWords * kGroup + (j * kWords + w % kWords) * 8;
}

// One row's codes of a block, as a lane holds them.
template <int kGroup>
__device__ __forceinline__ void load_codes(uint32_t (&w)[4], const uint8_t* row, int e0, int E, int j) {
  constexpr int kWords = kGroup / 32;
#pragma unroll
  for (int i = 0; i < 4; i += kWords) {
    const int e = e0 + column_of<kGroup>(i, j);
    if (e < E) {
      const uint8_t* p = row + e / 2;
      if constexpr (kWords == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else if constexpr (kWords == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[i] = v.x; w[i + 1] = v.y;
      } else {
        w[i] = __ldg(reinterpret_cast<const uint32_t*>(p));
      }
    } else {
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[i + k] = 0;
    }
  }
}

template <int kGroup, int NT>
__global__ void __launch_bounds__(Proj<NT>::kWarps * 32, 2)
proj_w4_kernel(const ProjArgs a) {
  using L = Proj<NT>;
  constexpr int kWarps = L::kWarps, kDepth = L::kDepth;
  constexpr int kGroups = kColumns / kGroup;  // of a block
  constexpr int kWords = kGroup / 32;
  extern __shared__ float join[];  // [warp][row][token]
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int g = lane >> 2, j = lane & 3;
  const int n0 = blockIdx.x * L::kRows;
  const int64_t t0 = int64_t(blockIdx.y) * (8 * NT);
  const int tokens = static_cast<int>(min(a.T - t0, int64_t(8 * NT)));
  const int groups = a.E / kGroup;
  const int blocks = (a.E + kColumns - 1) / kColumns;
  // this lane's rows: g and g + 8; past the last: the last again
  const uint8_t* codes[2];
  int64_t at_group[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t n = min(n0 + h * 8 + g, a.N - 1);
    codes[h] = a.codes + n * (a.E / 2);
    at_group[h] = n * groups;
  }
  float total[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) total[t][i] = 0.0f;

  uint32_t w[kDepth][2][4];
  auto load = [&](uint32_t (&to)[2][4], int block) {
#pragma unroll
    for (int h = 0; h < 2; ++h) load_codes<kGroup>(to[h], codes[h], block * kColumns, a.E, j);
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (warp + d * kWarps < blocks) load(w[d], warp + d * kWarps);
#pragma unroll 1
  for (int b0 = warp; b0 < blocks; b0 += kWarps * kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int block = b0 + d * kWarps;
      if (block >= blocks) break;
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        const int group = block * kGroups + q;
        if (group >= groups) break;
        float scale[2];
        uint32_t z64[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          scale[h] = bf_lo(__ldg(a.scales + at_group[h] + group));
          const float z = a.zeros != nullptr ? static_cast<float>(__ldg(a.zeros + at_group[h] + group)) : 8.0f;
          z64[h] = pack2(z * -0.015625f, z * -0.015625f);
        }
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
#pragma unroll
        for (int v = 0; v < kWords; ++v) {
          const int i = q * kWords + v;
          const int e = block * kColumns + column_of<kGroup>(i, j);
          uint32_t c[2][4];  // [k step][operand register]
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) c[k][r] = code_pair(w[d][r & 1][i], 2 * k + (r >> 1), z64[r & 1]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (t * 8 + g < tokens) x = ldg16(a.x + (t0 + t * 8 + g) * a.x_stride + e);
            mma_bf16(acc[t], c[0], __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632));
            mma_bf16(acc[t], c[1], __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) total[t][i] = fmaf(scale[i >> 1], acc[t][i], total[t][i]);
      }
      if (block + kDepth * kWarps < blocks) load(w[d], block + kDepth * kWarps);
    }
  }

  // the warps' sums, in their order
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      join[(warp * L::kRows + (i >> 1) * 8 + g) * L::kPitch + t * 8 + 2 * j + (i & 1)] = total[t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < L::kRows * tokens; i += kWarps * 32) {
    const int row = i % L::kRows, t = i / L::kRows;
    if (n0 + row >= a.N) continue;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) sum += join[(k * L::kRows + row) * L::kPitch + t];
    a.out[(t0 + t) * a.N + n0 + row] = static_cast<ple_bf16_t>(pack2(64.0f * sum, 0.0f) & 0xffffu);
  }
}

template <int kGroup, int NT>
cudaError_t launch(const ProjArgs& a, cudaStream_t stream) {
  using L = Proj<NT>;
  static_assert(L::kSmem <= 48 << 10, "more would have to be asked for");
  const auto kernel = proj_w4_kernel<kGroup, NT>;
  const dim3 grid((a.N + L::kRows - 1) / L::kRows, static_cast<unsigned>((a.T + 8 * NT - 1) / (8 * NT)));
  return launch_kernel(kernel, grid, dim3(L::kWarps * 32), L::kSmem, stream, 1, a);
}

// ---------------------------------------------------------------------------
// Up to 64 tokens at a time: the 5th-generation tensor cores
// ---------------------------------------------------------------------------
// With this many tokens the warp-wide instructions would be the bound (a
// quarter of the rate, and every warp reading every x). A CTA takes 128 rows
// of W as the first operand, (c - z) / 64 in bf16 (exact), against the tokens,
// 128 columns to a stage. W goes through registers into tensor memory and x
// as it is into shared memory: with both laid out in shared memory its
// bandwidth was the bound (4096 x 16384, 64 tokens: 32 us). Now 24.5 us, 1.5
// TB/s. What bounds it is a stage's chain of waiting, unpacking, storing and
// handing over, at 53 % of the issue slots: of 13.3 M warp instructions a
// quarter unpacks (13 for 8 weights), the others copy x by 16 bytes, take out
// sums and wait.
// The sums of each group of columns get tensor-memory columns of their own,
// four sets in turn, and eight warps take them out, a row a thread, and add
// them up times the group's scale in float32.
// Where the rows alone would leave SMs without work, a cluster of CTAs shares
// a row tile: each takes part of the columns, and their sums meet through
// distributed shared memory, in the order of the CTAs.
//
// Warps: 0-15 lay out, 16 issues the products, 17-19 fetch scales and zero
// points, 20-27 take the sums, half of the tokens each four.
constexpr int kWideRows = 128;
constexpr int kLayWarps = 16, kSumWarps = 8;
constexpr int kWideThreads = (kLayWarps + 4 + kSumWarps) * 32;
constexpr int kMaxParts = 4;
constexpr int kSets = 4;  // of sums in tensor memory
constexpr int kParamSets = 4, kParamGroups = 4;  // groups' scales and zero points, a few groups at a time

template <int kTokens>
struct Wide {
  static constexpr int kX = kTokens * kColumns * 2;  // bytes of a stage's tokens
  static constexpr int kStages = 4;                  // of weights in tensor memory
  static constexpr int kXStages = 12;                // of tokens in shared memory
  static constexpr int kAhead = kXStages - kStages;  // as many stages ahead tokens are asked for
  static constexpr int kTmemW = kSets * kTokens;     // weights stand behind the sums
  static constexpr int kTmem = 512;                  // columns
  static constexpr int kAtParams = kXStages * kX;
  static constexpr int kAtBars = kAtParams + kParamSets * kParamGroups * kWideRows * 4;
  static constexpr int kAtWords = kAtBars + (2 * kStages + 2 * kSets + 2 * kParamSets + 1) * 8;
  static constexpr int kSmem = kAtWords + 16 + 1024;   // and alignment
  static_assert(kTmemW + kStages * kColumns / 2 <= kTmem, "tensor memory");
  static_assert(kTokens * kWideRows * 4 <= kXStages * kX, "the sums of a tile fit where the tokens were");
};

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 bytes to shared memory, or as many zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ float4 read_cluster(uint32_t at, uint32_t rank) {
  uint32_t there;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(there) : "memory");
  return v;
}

template <int kGroup, int kTokens>
__global__ void __launch_bounds__(kWideThreads, 1)
proj_w4_wide_kernel(const ProjArgs a, int parts, int32_t* dev_err) {
  using L = Wide<kTokens>;
  constexpr int kGroups = kColumns / kGroup;            // of a stage
  constexpr int kParamStages = kParamGroups / kGroups;  // of a set of scales and zero points
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem), bar0 = base + L::kAtBars;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto free = [&](int s) { return bar0 + 8u * (L::kStages + s); };
  auto sums_full = [&](int s) { return bar0 + 8u * (2 * L::kStages + s); };
  auto sums_free = [&](int s) { return bar0 + 8u * (2 * L::kStages + kSets + s); };
  auto params_full = [&](int s) { return bar0 + 8u * (2 * L::kStages + 2 * kSets + s); };
  auto params_free = [&](int s) { return bar0 + 8u * (2 * L::kStages + 2 * kSets + kParamSets + s); };
  const uint32_t done = bar0 + 8u * (2 * L::kStages + 2 * kSets + 2 * kParamSets);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kAtWords);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + L::kAtWords + 4);
  const int warp = threadIdx.x / 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full(s), kLayWarps / 2);
      mbar_init(free(s), 1);
    }
    for (int s = 0; s < kSets; ++s) {
      mbar_init(sums_full(s), 1);
      mbar_init(sums_free(s), kSumWarps);
    }
    for (int s = 0; s < kParamSets; ++s) {
      mbar_init(params_full(s), 1);
      mbar_init(params_free(s), (kParamStages == 1 ? kLayWarps / 2 : kLayWarps) + kSumWarps);
    }
    mbar_init(done, 1);
    mbar_fence_init();
    *abort_flag = 0;
  }
  if (warp == kLayWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(L::kTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const int part = blockIdx.x % parts;
  const int n0 = blockIdx.x / parts * kWideRows;
  const int64_t t0 = int64_t(blockIdx.y) * kTokens;
  const int tokens = static_cast<int>(min(a.T - t0, int64_t(kTokens)));
  const int groups = a.E / kGroup;
  // this part's stages of columns, cut between sets of scales where there are enough
  const int stages = (a.E + kColumns - 1) / kColumns, unit = stages >= parts * kParamStages ? kParamStages : 1;
  const int cuts = (stages + unit - 1) / unit;
  const int first = static_cast<int>(int64_t(part) * cuts / parts) * unit;
  const int last = min(static_cast<int>(int64_t(part + 1) * cuts / parts) * unit, stages);
  auto gave_up = [&](bool ok) {
    if (!ok) {
      *abort_flag = 1;
      set_dev_err(dev_err, PLE_DEVERR_TIMEOUT);
    }
    return !ok;
  };
  uint32_t* const params = reinterpret_cast<uint32_t*>(smem + L::kAtParams);  // [set][group][row]: scale, -z / 64
  float* const mine = reinterpret_cast<float*>(smem);  // a part's sums, [token][row]: where the operands were

  if (warp < kLayWarps) {
    // ---------------- operands ----------------
    // Two teams of eight warps, every other stage each. W: half of a row's
    // columns a thread, through registers into tensor memory. x: a chunk of 8
    // columns of every 16th token, copied to where the products read it.
    // Nothing is read past a row's end, nor of tokens that are not there:
    // zeros stand for both.
    const int team = warp / 8, row = threadIdx.x % kWideRows, half = threadIdx.x / kWideRows % 2;
    const uint8_t* const codes = a.codes + min(n0 + row, a.N - 1) * int64_t(a.E / 2) + half * 32;
    const uint32_t to_w = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + L::kTmemW + half * 32;
    const int chunk = threadIdx.x % 16, token0 = threadIdx.x / 16 % 16;
    const ple_bf16_t* const x = a.x + (t0 + token0) * a.x_stride + chunk * 8;
    auto fetch_w = [&](uint4 (&w)[2], int stage) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (stage < last && stage * kColumns + half * 64 + i * 32 < a.E)
          w[i] = __ldg(reinterpret_cast<const uint4*>(codes + int64_t(stage) * (kColumns / 2)) + i);
      }
    };
    auto fetch_x = [&](int stage) {
      if (stage < last) {
        const uint32_t to = base + (stage - first) % L::kXStages * L::kX + chunk_at(kTokens, token0, chunk);
        const ple_bf16_t* from = x + int64_t(stage) * kColumns;
        const bool in_row = stage * kColumns + chunk * 8 < a.E;
#pragma unroll
        for (int i = 0; i < kTokens / 16; ++i) {
          const bool there = token0 + 16 * i < tokens && in_row;
          copy16(to + i * 16 * 128, there ? from : a.x, there);
          from += 16 * a.x_stride;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint4 w[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) fetch_w(w[u], first + team + 2 * u);
    for (int k = first + team; k < first + L::kAhead; k += 2) fetch_x(k);
    bool ok = true;
#pragma unroll 1
    for (int k0 = first + team, round = 0; ok && k0 < last; k0 += L::kStages, ++round) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = k0 + 2 * u, s = team + 2 * u;
        if (k >= last) break;
        const int rel = (k - first) * kGroups, chunk_no = rel / kParamGroups;
        ok = wait_for(params_full(chunk_no % kParamSets), chunk_no / kParamSets & 1, abort_flag);
        // the products of kStages ago: their weights' place, and the tokens' that are asked for next
        ok = __all_sync(0xffffffffu, ok && wait_for(free(s), (round & 1) ^ 1u, abort_flag));
        if (!ok) break;
        fetch_x(k + L::kAhead);
        fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int group = (rel + (half * 64 + i * 32) / kGroup) % (kParamSets * kParamGroups);
          const uint32_t z64 = __byte_perm(params[group * kWideRows + row], 0, 0x1010);
          const uint32_t words[4] = {w[u][i].x, w[u][i].y, w[u][i].z, w[u][i].w};
          uint32_t v[16];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pair[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) pair[j] = code_pair(words[q], j, z64);
            v[4 * q] = __byte_perm(pair[0], pair[1], 0x5410);
            v[4 * q + 1] = __byte_perm(pair[2], pair[3], 0x5410);
            v[4 * q + 2] = __byte_perm(pair[0], pair[1], 0x7632);
            v[4 * q + 3] = __byte_perm(pair[2], pair[3], 0x7632);
          }
          tmem_store16(to_w + s * (kColumns / 2) + i * 16, v);
        }
        fetch_w(w[u], k + L::kStages);
        asm volatile("cp.async.wait_group %0;" ::"n"(L::kAhead / 2) : "memory");
        tmem_stored();
        fence_before();
        fence_operands();
        warp_arrive(full(s));
        // the last of a team's stages with these scales and zero points
        if (kParamStages == 1 || (k - first) % kParamStages >= kParamStages - 2) warp_arrive(params_free(chunk_no % kParamSets));
      }
    }
    gave_up(ok);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kLayWarps) {
    // ---------------- products ----------------
    const uint32_t acc = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t x_op = operand(base);
    int set = 0;
    uint32_t set_parity = 1;
    bool ok = true;
#pragma unroll 1
    for (int k = first; ok && k < last; ++k) {
      const int s = (k - first) % L::kStages, round = (k - first) / L::kStages;
      ok = __all_sync(0xffffffffu, wait_for(full(s), round & 1, abort_flag));
      if (!ok) break;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (k * kGroups + g >= groups) break;
        ok = __all_sync(0xffffffffu, wait_for(sums_free(set), set_parity, abort_flag));
        if (!ok) break;
        fence_after();
        if (elected()) {
          const uint32_t d = acc + set * kTokens, w = acc + L::kTmemW + s * (kColumns / 2), xm = x_op + (k - first) % L::kXStages * (L::kX >> 4);
#pragma unroll
          for (int i = 0; i < kGroup / 16; ++i) {
            const int step = g * (kGroup / 16) + i;
            mma_tmem(d, w + 8 * step, xm + (((step / 4) * kTokens * 128 + (step % 4) * 32) >> 4), idesc(kTokens, 1), i > 0);
          }
          mma_commit(sums_full(set));
        }
        __syncwarp();
        if (++set == kSets) { set = 0; set_parity ^= 1u; }
      }
      if (!ok) break;
      if (elected()) mma_commit(free(s));
      __syncwarp();
    }
    // however the loop ended, no product reads or writes after this
    if (elected()) mma_commit(done);
    __syncwarp();
    ok = wait_for(done, 0, nullptr) && ok;
    gave_up(ok);
  } else if (warp < kLayWarps + 4) {
    // ---------------- scales and zero points ----------------
    // A few bytes of every row: three warps take turns at fetching them
    // ahead, four groups of a row in one piece where that is aligned.
    const int chunks = ((last - first) * kGroups + kParamGroups - 1) / kParamGroups;
    const bool whole = groups % kParamGroups == 0 && first * kGroups % kParamGroups == 0 && (reinterpret_cast<uintptr_t>(a.scales) & 7) == 0 &&
                       (reinterpret_cast<uintptr_t>(a.zeros) & 3) == 0;
#pragma unroll 1
    for (int c = warp - (kLayWarps + 1); c < chunks; c += 3) {
      const int group0 = first * kGroups + c * kParamGroups;
      uint2 scales[kWideRows / 32];
      uint32_t zeros[kWideRows / 32];
#pragma unroll
      for (int i = 0; i < kWideRows / 32; ++i) {
        const int64_t at = min(int64_t(n0) + i * 32 + (threadIdx.x & 31), int64_t(a.N - 1)) * groups;
        zeros[i] = 0x08080808u;
        if (whole) {
          scales[i] = __ldg(reinterpret_cast<const uint2*>(a.scales + at + group0));
          if (a.zeros != nullptr) zeros[i] = __ldg(reinterpret_cast<const uint32_t*>(a.zeros + at + group0));
        } else {
          uint32_t v[kParamGroups], z[kParamGroups];
#pragma unroll
          for (int g = 0; g < kParamGroups; ++g) {
            const int64_t from = at + min(group0 + g, groups - 1);
            v[g] = __ldg(a.scales + from);
            z[g] = a.zeros != nullptr ? __ldg(a.zeros + from) : 8;
          }
          scales[i] = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
          zeros[i] = z[0] | z[1] << 8 | z[2] << 16 | z[3] << 24;
        }
      }
      if (gave_up(__all_sync(0xffffffffu, wait_for(params_free(c % kParamSets), c / kParamSets & 1 ^ 1, abort_flag)))) break;
#pragma unroll
      for (int i = 0; i < kWideRows / 32; ++i)
#pragma unroll
        for (int g = 0; g < kParamGroups; ++g) {
          const uint32_t two = g < 2 ? scales[i].x : scales[i].y;
          params[(c % kParamSets * kParamGroups + g) * kWideRows + i * 32 + (threadIdx.x & 31)] =
              (g % 2 == 0 ? two << 16 : two & 0xffff0000u) | pack2(static_cast<float>(zeros[i] >> (8 * g) & 0xff) * -0.015625f, 0.0f);
        }
      warp_arrive(params_full(c % kParamSets));
    }
  } else {
    // ---------------- sums: a row and half of the tokens a thread ----------------
    constexpr int kMine = kTokens / 2;
    const int t_first = (warp - kLayWarps - 4) / 4 * kMine;
    const int row = threadIdx.x % kWideRows;
    const int64_t n = min(n0 + row, a.N - 1);
    const int g0 = first * kGroups, g1 = min(last * kGroups, groups);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float total[kMine];
#pragma unroll
    for (int t = 0; t < kMine; ++t) total[t] = 0.0f;
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      const int set = (g - g0) % kSets, round = (g - g0) / kSets;
      const int chunk_no = (g - g0) / kParamGroups;
      if ((g - g0) % kParamGroups == 0 &&
          gave_up(__all_sync(0xffffffffu, wait_for(params_full(chunk_no % kParamSets), chunk_no / kParamSets & 1, abort_flag)))) break;
      const float scale = bf_hi(params[(g - g0) % (kParamSets * kParamGroups) * kWideRows + row]);
      if (gave_up(__all_sync(0xffffffffu, wait_for(sums_full(set), round & 1, abort_flag)))) break;
      fence_after();
#pragma unroll
      for (int q = 0; q < kMine / 16; ++q) {
        float v[16];
        tmem_load16(tmem + lanes + set * kTokens + t_first + 16 * q, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) total[16 * q + i] = fmaf(scale, v[i], total[16 * q + i]);
      }
      fence_before();
      warp_arrive(sums_free(set));
      if ((g - g0 + 1) % kParamGroups == 0) warp_arrive(params_free(chunk_no % kParamSets));
    }
    // all products are done, so their operands may be written over
    if (parts > 1) {
#pragma unroll
      for (int t = 0; t < kMine; ++t) mine[(t_first + t) * kWideRows + row] = total[t];
    } else if (n0 + row < a.N) {
#pragma unroll
      for (int t = 0; t < kMine; ++t)
        if (t_first + t < tokens) a.out[(t0 + t_first + t) * a.N + n] = static_cast<ple_bf16_t>(pack2(64.0f * total[t], 0.0f) & 0xffffu);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kLayWarps) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::kTmem) : "memory");
  }
  if (parts == 1) return;
  // the parts' sums, in their order, tokens shared out
  cluster_barrier();
  for (int i = threadIdx.x; part + i / (kWideRows / 4) * parts < tokens; i += kWideThreads) {
    const int t = part + i / (kWideRows / 4) * parts, row = i % (kWideRows / 4) * 4;
    float4 v[kMaxParts];
#pragma unroll
    for (int r = 0; r < kMaxParts; ++r)
      if (r < parts) v[r] = read_cluster(base + (t * kWideRows + row) * 4, r);
    float sum[4] = {};
#pragma unroll
    for (int r = 0; r < kMaxParts; ++r)
      if (r < parts) {
        sum[0] += v[r].x; sum[1] += v[r].y; sum[2] += v[r].z; sum[3] += v[r].w;
      }
#pragma unroll
    for (int m = 0; m < 4; ++m)
      if (n0 + row + m < a.N) a.out[(t0 + t) * a.N + n0 + row + m] = static_cast<ple_bf16_t>(pack2(64.0f * sum[m], 0.0f) & 0xffffu);
  }
  cluster_barrier();  // no CTA leaves while its sums are read
}

template <int kGroup, int kTokens>
cudaError_t launch_wide(const ProjArgs& a, int32_t* dev_err, cudaStream_t stream) {
  using L = Wide<kTokens>;
  const auto kernel = proj_w4_wide_kernel<kGroup, kTokens>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (err != cudaSuccess) return err;
  const int tiles = (a.N + kWideRows - 1) / kWideRows, stages = (a.E + kColumns - 1) / kColumns;
  const int blocks = static_cast<int>((a.T + kTokens - 1) / kTokens);
  // parts of the columns, as long as all CTAs are on SMs at once and have some stages each
  int parts = 1;
  while (parts < kMaxParts && int64_t(tiles) * blocks * parts * 2 <= num_sms() && stages >= parts * 2 * 2) parts *= 2;
  const dim3 grid(static_cast<unsigned>(tiles * parts), static_cast<unsigned>(blocks));
  return launch_kernel(kernel, grid, dim3(kWideThreads), L::kSmem, stream, static_cast<unsigned>(parts), a, parts, dev_err);
}

// Warp-wide instructions or the tensor cores of the 5th generation. The former
// are slower per token, the latter cost 6 us before the first sum is out (both
// operands laid out, tensor memory, the parts' sums). What decides is how many
// tokens there are and how often the first kernel's CTAs, 16 rows each, two an
// SM, fill the GPU. Measured, warp-wide / tensor cores, us, tokens over
// columns x rows:
//   16   4096 x 4096  7.0 / 11.6   8192 x 8192  25.1 / 26.6   4096 x 16384  25.9 / 20.5
//   24   2048 x 2048  4.3 /  8.4   4096 x 4096   9.2 / 11.5   4096 x  6144  16.9 / 16.3
//   64   2048 x 2048  8.7 /  9.6   4096 x 4096  20.4 / 12.9
// Hence up to 8 tokens always the first, up to 16 if its CTAs fill the GPU
// three times at most, up to 32 once at most, and more never.
template <int kGroup>
cudaError_t launch_tiles(const ProjArgs& a, int32_t* dev_err, cudaStream_t stream) {
  const int fills = (a.N - 1) / (Proj<1>::kRows * 2 * num_sms());  // beyond the first
  if (a.T <= 8) return launch<kGroup, 1>(a, stream);
  if (a.T <= 16 && fills < 3) return launch<kGroup, 2>(a, stream);
  if (a.T <= 32) return fills < 1 ? launch<kGroup, 4>(a, stream) : launch_wide<kGroup, 32>(a, dev_err, stream);
  return launch_wide<kGroup, 64>(a, dev_err, stream);
}

}  // namespace
}  // namespace ple

using namespace ple;

PLE_EXPORT ple_status ple_proj_w4(const ple_bf16_t* x, int64_t x_stride, int64_t num_tokens,
                                  int32_t in_dim, int32_t out_dim, const uint8_t* codes,
                                  const ple_bf16_t* scales, const uint8_t* zeros, int32_t group,
                                  ple_bf16_t* out, int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_proj_w4";
  if (num_tokens < 0 || num_tokens > INT32_MAX || in_dim < 1 || out_dim < 1)
    return fail(PLE_ERR_INVALID_ARG, "%s: num_tokens %lld, in_dim %d, out_dim %d", name,
                static_cast<long long>(num_tokens), in_dim, out_dim);
  if (group != 32 && group != 64 && group != 128)
    return fail(PLE_ERR_UNSUPPORTED, "%s: group %d (32, 64 or 128)", name, group);
  if (in_dim % group != 0)
    return fail(PLE_ERR_UNSUPPORTED, "%s: in_dim %d is not a multiple of the group %d", name, in_dim, group);
  if (num_tokens == 0) return PLE_OK;
  if (num_tokens > 65535 * 64)  // the grid's second dimension
    return fail(PLE_ERR_UNSUPPORTED, "%s: %lld tokens", name, static_cast<long long>(num_tokens));
  if (x == nullptr || codes == nullptr || scales == nullptr || out == nullptr)
    return fail(PLE_ERR_INVALID_ARG, "%s: null x, codes, scales or out", name);
  if (rows_overlap({out, 1, 0, num_tokens * out_dim * 2}, {x, num_tokens, x_stride * 2, int64_t(in_dim) * 2}))
    return fail(PLE_ERR_INVALID_ARG, "%s: out overlaps x", name);
  if (!aligned16(x) || !aligned16(codes) || x_stride % 8 != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: x and codes must be 16-byte aligned, x_stride a multiple of 8", name);
  const ProjArgs a{x, x_stride, num_tokens, in_dim, out_dim, codes, scales, zeros, out};
  return check_cuda(group == 128 ? launch_tiles<128>(a, dev_err, stream) : group == 64 ? launch_tiles<64>(a, dev_err, stream)
                                                                             : launch_tiles<32>(a, dev_err, stream), name);
}
