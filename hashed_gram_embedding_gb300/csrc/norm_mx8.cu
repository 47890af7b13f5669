// ple_norm_mx8: the residual's addition and the root-mean-square norm with
// its result in 8 bits, one pass over the data; ple_mx8_read: values of an
// 8-bit tensor.
//
//   s = x + residual, n = s / sqrt(mean(s^2) + eps) * gamma, mx8(n)
//
// Bound by memory: 2 bytes each of x, the residual and the sum, and 33 / 32
// of the result. A row stays in registers as float32, 8 neighbouring elements
// a thread and turn, so that loads and stores are wide; four lanes hold a
// block of 32 and agree on its scale by two shuffles; narrow rows share a CTA.
// The norm is taken of the float32 sum, not of the bf16 that sum_out gets: the
// rounding to 8 bits is the only one of the result. 16 elements a thread (32
// past 8192 columns), in pairs, two an instruction: with 8 the joining of the
// warps' sums took more instructions than the elements (8192 x 4096 with a
// residual 52.0 us then).
// Where each CTA would have more than four rows, CTAs stay and ask for their
// next row while they have one: 8192 x 4096 38.9 us (6.1 TB/s, 0.89 of the copy
// rate; 44.6 with a CTA a row), 2000 x 8192 22.6 (28.7). Fewer rows are dealt
// out as CTAs end, by a kernel with room for half as many threads more an SM:
// 3001 x 2176 7.6 (11.6 staying), 1024 x 4096 7.4, one row 3.4: a launch, a
// trip to memory and a barrier.
// ple_mx8_read takes two rows a thread in flight and stores whole sectors:
// 8192 x 4096 17.2 us (5.9 TB/s; 22.0 with one and 16-byte stores).
#include "mx8.cuh"

#include <cmath>

namespace ple {
namespace {

struct NormArgs {
  const ple_bf16_t *x, *residual, *gamma;
  int64_t x_stride, residual_stride, sum_stride;
  int64_t rows;
  int C;
  float eps;
  ple_bf16_t* sum_out;
  uint8_t *codes, *scales;
};

// A value for all threads of a row, in an order that the sizes alone decide;
// `none` changes nothing in a join. All threads of a CTA come by. (Barriers of
// their own for its rows, up to 16 of them, left an SM fewer CTAs: 3001 x 2176
// 10.4 us against 7.6.)
template <typename T, typename F>
__device__ __forceinline__ T over_row(T v, T* room, T none, F join) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  if (warps == 1) return v;
  if (lane == 0) room[warp] = v;
  __syncthreads();
  v = lane < warps ? room[lane] : none;
  for (int o = warps > 8 ? 8 : warps > 4 ? 4 : warps > 2 ? 2 : 1; o > 0; o >>= 1)
    v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  return __shfl_sync(0xffffffffu, v, 0);
}

// Values are held in pairs: two float32 operations an instruction.
__device__ __forceinline__ void unpack_pairs(uint4 w, uint64_t (&v)[4]) {
  v[0] = f2(bf_lo(w.x), bf_hi(w.x));
  v[1] = f2(bf_lo(w.y), bf_hi(w.y));
  v[2] = f2(bf_lo(w.z), bf_hi(w.z));
  v[3] = f2(bf_lo(w.w), bf_hi(w.w));
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
  float a, b;
  f2_split(v, a, b);
  return pack2(a, b);
}
// Largest magnitude of eight values; NaN if one is.
__device__ __forceinline__ float largest(const uint64_t (&v)[4]) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_split(v[i], x[2 * i], x[2 * i + 1]);
  return abs_max(abs_max(abs_max(x[0], x[1], x[2]), x[3], x[4]), abs_max(x[5], x[6], x[7]), 0.0f);
}

template <int kTurns, bool kMany, bool kAdds>
__global__ void __launch_bounds__(512, kTurns == 4 ? 1 : kMany ? 2 : 3)
norm_mx8_kernel(const NormArgs a) {
  __shared__ float sums[2][16];
  __shared__ uint32_t tops[16];
  __shared__ float again[16];
  pdl_wait();
  pdl_trigger();
  const int at = threadIdx.y * (blockDim.x / 32);  // this row's places in them
  const int64_t step = int64_t(gridDim.x) * blockDim.y;
  // Columns are a multiple of 128: whole groups of 16 lanes take part. In
  // every turn but the last they all do (the last may end inside a warp).
  const int c0 = threadIdx.x * 8, turn_columns = blockDim.x * 8;
  const bool all = c0 + (kTurns - 1) * turn_columns < a.C;
  auto in = [&](int t) { return t < kTurns - 1 ? c0 + t * turn_columns < a.C : all; };
  auto ask = [&](int64_t row, const ple_bf16_t* from, int64_t stride, uint4 (&to)[kTurns]) {
    const ple_bf16_t* const at_row = from + row * stride + c0;
    const bool there = row < a.rows;
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      to[t] = make_uint4(0, 0, 0, 0);
      if (there && in(t)) to[t] = *reinterpret_cast<const uint4*>(at_row + t * turn_columns);
    }
  };
  const float inv_c = 1.0f / static_cast<float>(a.C);
  // One row for each threadIdx.y, from `first` on, out of x (and the residual);
  // `ahead` rows on the next ones are asked for in their place.
  auto norm = [&](int64_t first, int turn, uint4 (&next)[kTurns], uint4 (&next_add)[kTurns], int64_t ahead) {
    const int64_t row = first + threadIdx.y;
    const bool live = row < a.rows;  // a CTA's last rows may not exist: zeros
    uint64_t v[kTurns][4];
    uint64_t squares = 0;  // a pair of zeros
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      unpack_pairs(next[t], v[t]);
      if constexpr (kAdds) {
        uint64_t r[4];
        unpack_pairs(next_add[t], r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[t][i] = f2_add(v[t][i], r[i]);
      }
    }
    if constexpr (kMany) {  // (what a row writes in place is its own)
      ask(row + ahead, a.x, a.x_stride, next);
      if constexpr (kAdds) ask(row + ahead, a.residual, a.residual_stride, next_add);
    }
    ple_bf16_t* const sum_row = a.sum_out + row * a.sum_stride + c0;
    const bool stores = a.sum_out != nullptr && live;
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      if (stores && in(t))
        *reinterpret_cast<uint4*>(sum_row + t * turn_columns) =
            make_uint4(pack_pair(v[t][0]), pack_pair(v[t][1]), pack_pair(v[t][2]), pack_pair(v[t][3]));
#pragma unroll
      for (int i = 0; i < 4; ++i) squares = f2_fma(v[t][i], v[t][i], squares);
    }
    const auto plus = [](float p, float q) { return p + q; };
    const auto both = [](uint64_t p) {
      float lo, hi;
      f2_split(p, lo, hi);
      return lo + hi;
    };
    float sum = over_row(both(squares), sums[turn] + at, 0.0f, plus);
    const float mean = fmaf(sum, inv_c, a.eps);
    float by = rsqrtf(mean);
    // a step of Newton's: the quotient's own rounding is left (an infinite sum makes zeros, and keeps them)
    if (by > 0.0f) by = by * fmaf(-0.5f * mean * by, by, 1.5f);
    // (3e38: an eps near float32's largest, with which the mean may leave it)
    const bool far = live && (!(sum < 1e38f && mean < 3e38f) || (sum < 1e-28f && a.eps < 1e-18f));
    if (blockDim.y > 1 && blockDim.x > 32 ? __syncthreads_or(far) : far) {
      // squares that leave float32: the row in units of a power of two near its
      // largest value (infinities and NaN stay what they are, and so do other
      // rows of the CTA)
      uint32_t top = 0;
#pragma unroll
      for (int t = 0; t < kTurns; ++t) top = max(top, abs_bits(largest(v[t])));
      top = over_row(top, tops + at, 0u, [](uint32_t p, uint32_t q) { return max(p, q); });
      const bool mine = far && top < 0x7F800000u && top > 0;
      const float unit = mine ? __uint_as_float(min(max(254 - static_cast<int>(top >> 23), 1), 253) << 23) : 1.0f;
      squares = 0;
#pragma unroll
      for (int t = 0; t < kTurns; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[t][i] = f2_mul(v[t][i], f2(unit, unit));
          squares = f2_fma(v[t][i], v[t][i], squares);
        }
      sum = over_row(both(squares), again + at, 0.0f, plus);
      if (mine) by = static_cast<float>(1.0 / sqrt(static_cast<double>(sum) / a.C + static_cast<double>(a.eps) * unit * unit));
    }
    uint8_t* const code_row = a.codes + row * a.C + c0;
    uint8_t* const scale_row = a.scales + mx_scale_at(row, c0 / kMxBlock, a.C);  // a turn is so many pieces on
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[t][i] = f2_mul(v[t][i], f2(by, by));
      if (a.gamma != nullptr) {
        uint64_t g[4];
        unpack_pairs(in(t) ? ldg16(a.gamma + c0 + t * turn_columns) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[t][i] = f2_mul(v[t][i], g[i]);
      }
      uint32_t top = abs_bits(largest(v[t]));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t b = mx_scale_byte(top);
      const float m = mx_inverse(b);
      // the bytes of the four blocks of a piece, in its first lane
      uint32_t word = b << (threadIdx.x / 4 % 4 * 8);
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      if (live && in(t)) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_split(f2_mul(v[t][i], f2(m, m)), y[2 * i], y[2 * i + 1]);
        *reinterpret_cast<uint2*>(code_row + t * turn_columns) =
            make_uint2(mx_codes4(y[0], y[1], y[2], y[3]), mx_codes4(y[4], y[5], y[6], y[7]));
        if (threadIdx.x % 16 == 0) *reinterpret_cast<uint32_t*>(scale_row + t * turn_columns / kMxTile * kMxPiece) = word;
      }
    }
  };
  const int64_t begin = int64_t(blockIdx.x) * blockDim.y;
  uint4 one[kTurns], two[kTurns];
  ask(begin + threadIdx.y, a.x, a.x_stride, one);
  if constexpr (kAdds) {
    ask(begin + threadIdx.y, a.residual, a.residual_stride, two);
    int turn = 0;
    for (int64_t first = begin; first < a.rows; first = kMany ? first + step : a.rows, turn ^= 1) norm(first, turn, one, two, step);
  } else if constexpr (kMany) {  // half the bytes a row: two rows ahead
    ask(begin + step + threadIdx.y, a.x, a.x_stride, two);
    for (int64_t first = begin; first < a.rows; first += 2 * step) {
      norm(first, 0, one, one, 2 * step);
      if (first + step < a.rows) norm(first + step, 1, two, two, 2 * step);
    }
  } else {
    norm(begin, 0, one, one, 0);
  }
}

template <int kTurns>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  const int threads = ((a.C / 8 + kTurns - 1) / kTurns + 31) / 32 * 32, at_once = threads <= 256 ? 256 / threads : 1;
  const int64_t need = (a.rows + at_once - 1) / at_once, most = int64_t(num_sms()) * (kTurns == 2 ? 1024 : 512) / (threads * at_once);
  const bool many = need > 4 * most;
  const bool adds = a.residual != nullptr;
  return launch_kernel(many ? adds ? norm_mx8_kernel<kTurns, true, true> : norm_mx8_kernel<kTurns, true, false>
                            : adds ? norm_mx8_kernel<kTurns, false, true> : norm_mx8_kernel<kTurns, false, false>,
                       dim3(static_cast<unsigned>(many ? most : need)), dim3(threads, at_once), 0, stream, 1, a);
}

// 16 codes a thread and row, of two rows at a time: a CTA takes 4096 columns.
__global__ void __launch_bounds__(256) mx8_read_kernel(const uint8_t* codes, const uint8_t* scales, int rows, int columns,
                                                       ple_bf16_t* out) {
  pdl_wait();
  pdl_trigger();
  const int c = (blockIdx.y * 256 + threadIdx.x) * 16;
  if (c >= columns) return;
  constexpr int kRows = 2;
  for (int64_t r0 = int64_t(blockIdx.x) * kRows; r0 < rows; r0 += int64_t(gridDim.x) * kRows) {
    uint4 w[kRows];
    uint32_t b[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (r0 + i < rows) {
        w[i] = __ldg(reinterpret_cast<const uint4*>(codes + (r0 + i) * columns + c));
        b[i] = __ldg(scales + mx_scale_at(r0 + i, c / kMxBlock, columns));
      }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (r0 + i < rows) {
        const float power = mx_power(b[i]);
        const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 f = mx_values2(words[k / 2] >> (k % 2 * 16) & 0xffff);
          v[k] = pack2(f.x * power, f.y * power);
        }
        store32(out + (r0 + i) * columns + c, v);
      }
  }
}

constexpr int kMaxNorm = 16384;  // columns: four turns of 512 threads

}  // namespace
}  // namespace ple

using namespace ple;

PLE_EXPORT size_t ple_mx8_scale_bytes(int64_t rows, int32_t columns) {
  const int64_t n = mx_scale_size(rows, columns);
  return n > 0 ? static_cast<size_t>(n) : 0;
}

PLE_EXPORT ple_status ple_norm_mx8(const ple_bf16_t* x, int64_t x_stride, const ple_bf16_t* residual,
                                   int64_t residual_stride, const ple_bf16_t* gamma, float eps,
                                   int64_t num_tokens, int32_t hidden, ple_bf16_t* sum_out,
                                   int64_t sum_stride, uint8_t* codes, uint8_t* scales,
                                   cudaStream_t stream) {
  const char* name = "ple_norm_mx8";
  if (num_tokens < 0 || num_tokens > INT32_MAX || hidden < 1 || !(eps > 0.0f) || !std::isfinite(eps))
    return fail(PLE_ERR_INVALID_ARG, "%s: num_tokens %lld, hidden %d, eps %g", name,
                static_cast<long long>(num_tokens), hidden, static_cast<double>(eps));
  if (hidden % kMxTile != 0 || hidden > kMaxNorm)
    return fail(PLE_ERR_UNSUPPORTED, "%s: hidden %d (a multiple of %d up to %d)", name, hidden, kMxTile, kMaxNorm);
  if (num_tokens == 0) return PLE_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr)
    return fail(PLE_ERR_INVALID_ARG, "%s: null x, codes or scales", name);
  if (!aligned16(x) || !aligned16(residual) || !aligned16(gamma) || !aligned16(sum_out) || !aligned16(codes) ||
      !aligned16(scales) || x_stride % 8 != 0 || residual_stride % 8 != 0 || sum_stride % 8 != 0)
    return fail(PLE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned, strides multiples of 8", name);
  const int64_t width = int64_t(hidden) * 2;
  const RowSpan in[] = {{x, num_tokens, x_stride * 2, width},
                        {residual, residual == nullptr ? 0 : num_tokens, residual_stride * 2, width},
                        {gamma, gamma == nullptr ? 0 : 1, 0, width}};
  const RowSpan out[] = {{codes, 1, 0, num_tokens * hidden},
                         {scales, 1, 0, mx_scale_size(num_tokens, hidden)},
                         {sum_out, sum_out == nullptr ? 0 : num_tokens, sum_stride * 2, width}};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 3; ++i) {
      // a row is read whole before its place is written
      const bool itself = o == 2 && i < 2 && out[o].base == in[i].base && out[o].stride == in[i].stride;
      if (!itself && rows_overlap(out[o], in[i]))
        return fail(PLE_ERR_INVALID_ARG, "%s: an output overlaps an input", name);
    }
    for (int i = 0; i < o; ++i)
      if (rows_overlap(out[o], out[i])) return fail(PLE_ERR_INVALID_ARG, "%s: two outputs overlap", name);
  }
  if (sum_out != nullptr && num_tokens > 1 && (sum_stride < 0 ? -sum_stride : sum_stride) < hidden)
    return fail(PLE_ERR_INVALID_ARG, "%s: rows of sum_out overlap", name);
  const NormArgs a{x, residual, gamma, x_stride, residual_stride, sum_stride, num_tokens, hidden, eps, sum_out, codes, scales};
  return check_cuda(hidden > 8192 ? launch_norm<4>(a, stream) : launch_norm<2>(a, stream), name);
}

PLE_EXPORT ple_status ple_mx8_read(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t columns,
                                   ple_bf16_t* out, cudaStream_t stream) {
  const char* name = "ple_mx8_read";
  if (rows < 0 || rows > INT32_MAX || columns < 1)
    return fail(PLE_ERR_INVALID_ARG, "%s: rows %lld, columns %d", name, static_cast<long long>(rows), columns);
  if (columns % kMxTile != 0 || columns > 65535 * 4096)  // the grid's second dimension
    return fail(PLE_ERR_UNSUPPORTED, "%s: columns %d (a multiple of %d)", name, columns, kMxTile);
  if (rows == 0) return PLE_OK;
  if (codes == nullptr || scales == nullptr || out == nullptr)
    return fail(PLE_ERR_INVALID_ARG, "%s: null codes, scales or out", name);
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out))
    return fail(PLE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", name);
  const size_t n = static_cast<size_t>(rows) * columns;
  if (overlaps(out, 2 * n, codes, n) || overlaps(out, 2 * n, scales, mx_scale_size(rows, columns)))
    return fail(PLE_ERR_INVALID_ARG, "%s: out overlaps codes or scales", name);
  const int across = (columns + 4095) / 4096;
  const int64_t most = (int64_t(num_sms()) * 32 + across - 1) / across, need = (rows + 1) / 2;
  return check_cuda(launch_kernel(mx8_read_kernel, dim3(static_cast<unsigned>(need < most ? need : most), across), dim3(256), 0,
                                  stream, 1, codes, scales, static_cast<int>(rows), columns, out), name);
}
