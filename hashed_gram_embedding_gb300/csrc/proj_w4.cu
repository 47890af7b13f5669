// ple_proj_w4: out = x W^T with W in 4 bits, a scale and a zero point per
// group of columns, for steps of few tokens.
//
// Bound by reading the codes, half a byte a weight. Products on warp-wide
// matrix instructions (16 x 8 x 16, bf16, f32 sums): W is the A operand, 16
// output rows, and 8 tokens fill the other side. A weight's code never meets
// memory again: masked out of its word where it stands, a pair of codes is a
// pair of bf16 subnormals (c 2^-133, or c 2^-129 for the upper half of a
// byte), and one fused multiply-add makes (c - z) / 64 of it, exactly. The
// scale meets the float32 sum once per group:
//   out[t][n] = sum_g 64 s_ng sum_{e in g} x_te (c_ne - z_ng) / 64.
// The contraction index may run in any order, so a lane reads codes in the
// widest pieces that lie in one group - 16, 8 or 4 bytes of a row for groups
// of 128, 64 or 32 columns, four lanes together a group of a row - and the
// x of the same columns, 16 bytes a word of codes.
//
// A CTA takes 16 MT output rows and all columns; its warps take blocks of 128
// columns in turn, each with the next blocks' codes in flight, and add their
// sums up in shared memory, in the warps' order. All codes of a small weight
// are thus asked for at once, by as many SMs as there are.
#include "common.cuh"

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
  static constexpr int kMT = NT >= 4 ? 2 : 1;      // tiles of 16 rows
  static constexpr int kWarps = 8;
  static constexpr int kDepth = NT >= 4 ? 2 : 4;   // blocks of codes in flight
  static constexpr int kRows = 16 * kMT;
  static constexpr int kPitch = 8 * NT + 1;        // floats of a row's sums, padded
  static constexpr int kJoin = NT == 8 ? kWarps / 2 : kWarps;  // warps whose sums are held at a time
  static constexpr int kSmem = kJoin * kRows * kPitch * 4;
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
  const uint32_t c = (i < 2 ? word : word >> 8) & (i % 2 == 0 ? 0x000F000Fu : 0x00F000F0u);
  uint32_t y;  // 2^127, or 2^123
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(c), "r"(i % 2 == 0 ? 0x7F007F00u : 0x7D007D00u), "r"(z64));
  return y;
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
__global__ void __launch_bounds__(Proj<NT>::kWarps * 32, NT >= 4 ? 1 : 2)
proj_w4_kernel(const ProjArgs a) {
  using L = Proj<NT>;
  constexpr int MT = L::kMT, kWarps = L::kWarps, kDepth = L::kDepth;
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
  // this lane's rows: g and g + 8 of each tile; past the last: the last again
  const uint8_t* codes[MT][2];
  int64_t at_group[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = min(n0 + m * 16 + h * 8 + g, a.N - 1);
      codes[m][h] = a.codes + n * (a.E / 2);
      at_group[m][h] = n * groups;
    }
  float total[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[m][t][i] = 0.0f;

  uint32_t w[kDepth][MT][2][4];
  auto load = [&](uint32_t (&to)[MT][2][4], int block) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) load_codes<kGroup>(to[m][h], codes[m][h], block * kColumns, a.E, j);
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
        float scale[MT][2];
        uint32_t z64[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            scale[m][h] = 64.0f * bf_lo(__ldg(a.scales + at_group[m][h] + group));
            const float z = a.zeros != nullptr ? static_cast<float>(__ldg(a.zeros + at_group[m][h] + group)) : 8.0f;
            z64[m][h] = pack2(z * -0.015625f, z * -0.015625f);
          }
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.0f;
#pragma unroll
        for (int v = 0; v < kWords; ++v) {
          const int i = q * kWords + v;
          const int e = block * kColumns + column_of<kGroup>(i, j);
          uint32_t c[MT][2][4];  // [tile][k step][operand register]
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                c[m][k][r] = code_pair(w[d][m][r & 1][i], 2 * k + (r >> 1), z64[m][r & 1]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (t * 8 + g < tokens) x = ldg16(a.x + (t0 + t * 8 + g) * a.x_stride + e);
            const uint32_t x0 = __byte_perm(x.x, x.z, 0x5410), x1 = __byte_perm(x.x, x.z, 0x7632);
            const uint32_t x2 = __byte_perm(x.y, x.w, 0x5410), x3 = __byte_perm(x.y, x.w, 0x7632);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma_bf16(acc[m][t], c[m][0], x0, x1);
              mma_bf16(acc[m][t], c[m][1], x2, x3);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[m][t][i] = fmaf(scale[m][i >> 1], acc[m][t][i], total[m][t][i]);
      }
      if (block + kDepth * kWarps < blocks) load(w[d], block + kDepth * kWarps);
    }
  }

  // the warps' sums, in their order
  auto place = [&](int slot, int m, int t, int i) -> float& {
    return join[(slot * L::kRows + m * 16 + (i >> 1) * 8 + g) * L::kPitch + t * 8 + 2 * j + (i & 1)];
  };
  if constexpr (L::kJoin < kWarps) {  // the upper half of the warps hands over first
    if (warp >= L::kJoin) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) place(warp - L::kJoin, m, t, i) = total[m][t][i];
    }
    __syncthreads();
    if (warp < L::kJoin) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) place(warp, m, t, i) = total[m][t][i] + place(warp, m, t, i);
    }
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) place(warp, m, t, i) = total[m][t][i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < L::kRows * tokens; i += kWarps * 32) {
    const int row = i % L::kRows, t = i / L::kRows;
    if (n0 + row >= a.N) continue;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < L::kJoin; ++k) sum += join[(k * L::kRows + row) * L::kPitch + t];
    a.out[(t0 + t) * a.N + n0 + row] = static_cast<ple_bf16_t>(pack2(sum, 0.0f) & 0xffffu);
  }
}

template <int kGroup, int NT>
cudaError_t launch(const ProjArgs& a, cudaStream_t stream) {
  using L = Proj<NT>;
  const auto kernel = proj_w4_kernel<kGroup, NT>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (err != cudaSuccess) return err;
  const dim3 grid((a.N + L::kRows - 1) / L::kRows, static_cast<unsigned>((a.T + 8 * NT - 1) / (8 * NT)));
  return launch_kernel(kernel, grid, dim3(L::kWarps * 32), L::kSmem, stream, 1, a);
}

// As many tiles of 8 tokens as the step has, up to 8: the codes are read once
// for each 64 tokens.
template <int kGroup>
cudaError_t launch_tiles(const ProjArgs& a, cudaStream_t stream) {
  return a.T <= 8 ? launch<kGroup, 1>(a, stream) : a.T <= 16 ? launch<kGroup, 2>(a, stream)
       : a.T <= 32 ? launch<kGroup, 4>(a, stream) : launch<kGroup, 8>(a, stream);
}

}  // namespace
}  // namespace ple

using namespace ple;

PLE_EXPORT ple_status ple_proj_w4(const ple_bf16_t* x, int64_t x_stride, int64_t num_tokens,
                                  int32_t in_dim, int32_t out_dim, const uint8_t* codes,
                                  const ple_bf16_t* scales, const uint8_t* zeros, int32_t group,
                                  ple_bf16_t* out, int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_proj_w4";
  (void)dev_err;
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
  if (!aligned16(x) || !aligned16(codes) || x_stride % 8 != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: x and codes must be 16-byte aligned, x_stride a multiple of 8", name);
  const ProjArgs a{x, x_stride, num_tokens, in_dim, out_dim, codes, scales, zeros, out};
  return check_cuda(group == 128 ? launch_tiles<128>(a, stream) : group == 64 ? launch_tiles<64>(a, stream)
                                                                             : launch_tiles<32>(a, stream), name);
}
