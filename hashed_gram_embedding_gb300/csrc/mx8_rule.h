// Which kernel takes a product of 8-bit tensors, and how many CTAs share its
// columns: arithmetic on sizes alone, so that it can be asked without a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace ple {

struct ProductSize {
  int64_t tokens;
  int columns, rows;  // of the result: of W, or half as many
  bool gated;
};

// Single CTAs by the tokens of their tile: how many share an SM, and how many
// a cluster may have.
constexpr int few_resident(int tile) { return tile <= 64 ? 2 : 1; }
constexpr int few_max_parts(int tile) { return few_resident(tile) == 2 ? 8 : 4; }

// Parts that a cluster cuts the columns into: as many as keep all CTAs on SMs
// at once and leave each some atoms.
inline int few_parts(int tile, int64_t ctas, int atoms, int sms) {
  int parts = 1;
  while (parts < few_max_parts(tile) && ctas * parts * 2 <= int64_t(sms) * few_resident(tile) && atoms >= parts * 2 * 4) parts *= 2;
  return parts;
}

// What a launch takes, in 10 ns, from measurements: by pairs of CTAs a stage
// of 256 columns 56, a tile's start and end 330, all else 480, and never less
// than W's way from memory at 5.2 TB/s and 600; by single ones
// an atom of 128 columns 41 (gated, 128 tokens: 70), a tile's start and end
// 800 (300, and 6 for each token: its sums are taken out and joined), all else
// 70.
inline int64_t time_of_pairs(const ProductSize& p, int64_t pairs) {
  const int rows = p.gated ? 128 : 256;
  const int64_t units = (p.tokens + 255) / 256 * ((p.rows + rows - 1) / rows);
  const int64_t w = int64_t(p.gated ? 2 : 1) * p.rows * p.columns;
  return std::max((units + pairs - 1) / pairs * ((p.columns / 128 + 1) / 2 * 56 + 330) + 480, w / 52000 + 600);
}
inline int64_t time_of_ctas(const ProductSize& p, int tile, int sms) {
  const int64_t ctas = (p.rows + 127) / 128 * ((p.tokens + tile - 1) / tile);
  const int atoms = p.columns / 128, parts = few_parts(tile, ctas, atoms, sms);
  const int64_t atom = p.gated ? 70 : 41, ends = p.gated ? 300 + 6 * p.tokens : 800;
  return (ctas * parts + sms - 1) / sms * ((atoms + parts - 1) / parts * atom + ends) + 70;
}

// Few tokens go to single CTAs, with a tile that holds them; many, in blocks of
// 256, stay there while pairs would leave too much of the GPU idle, and go to
// pairs otherwise. Measured, pairs / single CTAs, us, tokens over columns x
// rows:
//   200  4096 x 4096  15.8 / 11.7   300  8192 x 2048  25.3 / 15.1   400  2048 x 1024  11.0 / 10.3
//   512  4096 x 4096  16.7 / 15.6   512  2048 x 8192  12.9 / 15.3   768  4096 x 4096  17.2 / 20.6
//  1023  2048 x 8192  20.0 / 30.1  1024 16384 x 4096  47.9 / 56.9
// up to 128 tokens, where single CTAs always take them; pairs are 6 to 11 %
// faster past 152 tiles of rows, which is left at that:
//    32 4096 x 16384  19.8 / 15.5    64 16384 x 4096  45.1 / 17.4    64  2048 x 8192  11.0 /  8.4
//   128   512 x 8192   8.2 /  6.8   128  4096 x 4096  15.1 /  9.6   128 4096 x 16384  20.7 / 18.5
//   128 16384 x 4096  45.8 / 19.3   128 4096 x 20000  32.1 / 34.0   128 1024 x 32768  15.9 / 17.8
// gated:
//    33  4096 x 4096  16.0 / 11.6    48  2048 x 8192  12.7 / 12.7    64 4096 x 16384  32.2 / 29.3
//    80  2048 x 8192  12.4 / 14.4   112  4096 x 4096  16.5 / 15.8   112 4096 x 16384  32.5 / 32.9
//   150  4096 x 4096  16.5 / 19.3   256  2048 x 8192  13.1 / 20.8   512  4096 x  1024  14.4 / 15.4
// The tiles: 16 tokens are worth one of their own only gated, whose stages are
// twice as large (16 and 32 wide, one token 4096 x 16384 24.7 / 25.2; 16 tokens
// 4096 x 4096, not gated, 7.4 / 6.9), 64 only otherwise (64 and 128 wide, 64 tokens
// 16384 x 4096 17.3 / 17.8; gated 4096 x 4096 15.3 / 13.0).
//
// The tokens of a single CTA's tile, or 0: pairs. `pairs` says how many of these
// the GPU holds, and is asked only where it counts.
template <typename Pairs>
int product_tile(const ProductSize& p, int sms, Pairs pairs) {
  if (p.gated) {
    if (p.tokens <= 32) return p.tokens <= 16 ? 16 : 32;
    return p.tokens <= 128 && time_of_ctas(p, 128, sms) <= time_of_pairs(p, pairs()) ? 128 : 0;
  }
  if (p.tokens <= 128) return p.tokens <= 32 ? 32 : p.tokens <= 64 ? 64 : 128;
  return time_of_ctas(p, 256, sms) < time_of_pairs(p, pairs()) ? 256 : 0;
}

}  // namespace ple
