// ple_proj_mx8 and ple_gated_mx8: products of 8-bit tensors (mx8.cuh).
//
//   ple_proj_mx8    out = residual + x W^T, rounded once to bf16
//   ple_gated_mx8   h = act(x Wg^T) * (x Wu^T), quantised as it is computed
//
// One thread block takes 64 tokens and 64 rows of W (gated: 32 of the gate's
// and the 32 of the other half that meet them) and a block of 32 columns at a
// time, its values in shared memory as float32.
#include "mx8.cuh"

namespace ple {
namespace {

struct ProductArgs {
  const uint8_t *x, *x_scales, *w, *w_scales;
  int64_t T;
  int E, N;  // columns; rows of the result: of W, or half as many
  int gelu;
  const ple_bf16_t* residual;
  int64_t residual_stride;
  ple_bf16_t* out;
  uint8_t *codes, *scales;
};

__device__ __forceinline__ float activation(float g, int gelu) {
  const float turn = gelu ? 1.5957691216057308f * (g + 0.044715f * g * g * g) : g;  // 2 sqrt(2 / pi)
  return g / (1.0f + expf(-turn));
}

template <bool kGated>
__global__ void __launch_bounds__(256) product_kernel(const ProductArgs a) {
  __shared__ float xs[32][65], ws[32][65];
  const int64_t t0 = int64_t(blockIdx.y) * 64;
  const int n0 = blockIdx.x * (kGated ? 32 : 64);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  // this thread's 8 codes of x and of W
  const int r = threadIdx.x / 4, c = threadIdx.x % 4 * 8;
  const int64_t t = t0 + r;
  const int64_t n = kGated ? int64_t(r / 32) * a.N + n0 + r % 32 : n0 + r;
  const bool t_in = t < a.T, n_in = kGated || n < a.N;
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    uint2 cx = make_uint2(0, 0), cw = cx;
    float px = 0.0f, pw = 0.0f;
    if (t_in) {
      cx = __ldg(reinterpret_cast<const uint2*>(a.x + t * a.E + e0 + c));
      px = mx_power(a.x_scales[mx_scale_at(t, e0 / 32, a.E)]);
    }
    if (n_in) {
      cw = __ldg(reinterpret_cast<const uint2*>(a.w + n * a.E + e0 + c));
      pw = mx_power(a.w_scales[mx_scale_at(n, e0 / 32, a.E)]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 fx = mx_values2((i < 2 ? cx.x : cx.y) >> (i % 2 * 16) & 0xffff);
      const float2 fw = mx_values2((i < 2 ? cw.x : cw.y) >> (i % 2 * 16) & 0xffff);
      xs[c + 2 * i][r] = fx.x * px;
      xs[c + 2 * i + 1][r] = fx.y * px;
      ws[c + 2 * i][r] = fw.x * pw;
      ws[c + 2 * i + 1][r] = fw.y * pw;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
      float p[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = xs[k][ty * 4 + i];
        q[i] = ws[k][tx + 16 * i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(p[i], q[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t token = t0 + ty * 4 + i;
    if constexpr (kGated) {
      const float h0 = activation(acc[i][0], a.gelu) * acc[i][2], h1 = activation(acc[i][1], a.gelu) * acc[i][3];
      uint32_t top = max(abs_bits(h0), abs_bits(h1));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const uint32_t b = mx_scale_byte(top);
      if (token < a.T) {
        a.codes[token * a.N + n0 + tx] = static_cast<uint8_t>(mx_codes2(h0 * mx_inverse(b), 0.0f));
        a.codes[token * a.N + n0 + tx + 16] = static_cast<uint8_t>(mx_codes2(h1 * mx_inverse(b), 0.0f));
        if (tx == 0) a.scales[mx_scale_at(token, n0 / 32, a.N)] = static_cast<uint8_t>(b);
      }
    } else if (token < a.T) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = n0 + tx + 16 * j;
        if (row >= a.N) continue;
        float y = acc[i][j];
        if (a.residual != nullptr) y += bf_lo(a.residual[token * a.residual_stride + row]);
        a.out[token * a.N + row] = static_cast<ple_bf16_t>(pack2(y, 0.0f) & 0xffffu);
      }
    }
  }
}

ple_status check_product(const char* name, const uint8_t* x, const uint8_t* x_scales, int64_t num_tokens, int32_t in_dim,
                         const uint8_t* w, const uint8_t* w_scales, int32_t rows) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || in_dim < 1 || rows < 1)
    return fail(PLE_ERR_INVALID_ARG, "%s: %lld tokens, %d columns, %d rows", name, static_cast<long long>(num_tokens),
                in_dim, rows);
  if (in_dim % kMxTile != 0)
    return fail(PLE_ERR_UNSUPPORTED, "%s: %d columns (a multiple of %d)", name, in_dim, kMxTile);
  if (num_tokens == 0) return PLE_OK;
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
  const ProductArgs a{x, x_scales, w, w_scales, num_tokens, hidden, inner, activation == PLE_GELU, nullptr, 0, nullptr,
                      codes, scales};
  const size_t n = static_cast<size_t>(num_tokens) * inner, m = mx_scale_size(num_tokens, inner);
  if (meets_operands(codes, n, a, 2LL * inner) || meets_operands(scales, m, a, 2LL * inner) || overlaps(codes, n, scales, m))
    return fail(PLE_ERR_INVALID_ARG, "%s: an output overlaps an operand or the other output", name);
  const dim3 grid(inner / 32, static_cast<unsigned>((num_tokens + 63) / 64));
  return check_cuda(launch_kernel_pdl(false, product_kernel<true>, grid, dim3(256), 0, stream, 1, a), name);
}

PLE_EXPORT ple_status ple_proj_mx8(const uint8_t* x, const uint8_t* x_scales, int64_t num_tokens, int32_t in_dim,
                                   const uint8_t* w, const uint8_t* w_scales, int32_t out_dim,
                                   const ple_bf16_t* residual, int64_t residual_stride, ple_bf16_t* out,
                                   int32_t* dev_err, cudaStream_t stream) {
  const char* name = "ple_proj_mx8";
  const ple_status s = check_product(name, x, x_scales, num_tokens, in_dim, w, w_scales, out_dim);
  if (s != PLE_OK || num_tokens == 0) return s;
  if (out == nullptr) return fail(PLE_ERR_INVALID_ARG, "%s: null out", name);
  const ProductArgs a{x, x_scales, w, w_scales, num_tokens, in_dim, out_dim, 0, residual, residual_stride, out,
                      nullptr, nullptr};
  const size_t n = static_cast<size_t>(num_tokens) * out_dim * 2;
  if (meets_operands(out, n, a, out_dim)) return fail(PLE_ERR_INVALID_ARG, "%s: out overlaps an operand", name);
  if (residual != nullptr && !(residual == out && (residual_stride == out_dim || num_tokens == 1)) &&
      rows_overlap({out, 1, 0, static_cast<int64_t>(n)}, {residual, num_tokens, residual_stride * 2, int64_t(out_dim) * 2}))
    return fail(PLE_ERR_INVALID_ARG, "%s: out overlaps the residual and is not the residual", name);
  const dim3 grid((out_dim + 63) / 64, static_cast<unsigned>((num_tokens + 63) / 64));
  return check_cuda(launch_kernel_pdl(false, product_kernel<false>, grid, dim3(256), 0, stream, 1, a), name);
}
