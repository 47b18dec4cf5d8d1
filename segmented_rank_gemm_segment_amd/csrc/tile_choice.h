// Which kernel, in which tiles, a product with MXFP4 operands takes: host rules on
// the batch's sizes (plain C++, so that a test without a GPU can hold its shapes
// against them).
#pragma once

#include <cmath>
#include <cstdint>

#ifndef LORA_GEMM_192_COST
// Relative cost per output element of a 192 x 256 tile against a 256 x 256
// one (more LDS fragment reads per flop), in percent.
#define LORA_GEMM_192_COST 110
#endif

namespace lora {

constexpr int kCUs = 256;   // compute units of an MI355X

// Whether a large batch of M rows takes large tiles of 192 x 256: when their rounds
// of kCUs tiles cost less (rounds times tile area, the narrower tile charged its
// extra LDS traffic per flop).
inline bool large192_tiles(int M, int N) {
  const int64_t tn256 = (N + 255) / 256;
  const int64_t r256 = ((int64_t)(M + 255) / 256 * tn256 + kCUs - 1) / kCUs;
  const int64_t r192 = ((int64_t)(M + 191) / 192 * tn256 + kCUs - 1) / kCUs;
  return r192 * 192 * LORA_GEMM_192_COST < r256 * 256 * 100;
}

// kMxStream8, kMxStream16: streamed, that many rows at most (mx_stream.cuh);
// kMxTiles32, kMxTiles64: tiles of that many rows (mx_mid.cuh); kMxTiles128 and,
// with adapters, kMxTiles192 and kMxTiles256: the tiles of the bf16 product
// (gemm_tile.cuh); kMxPersistent: 256 x 256 tiles of the persistent kernels
// (mx_weight.cuh, mx_product.hip).
enum MxKernel {
  kMxStream8,
  kMxStream16,
  kMxTiles32,
  kMxTiles64,
  kMxTiles128,
  kMxTiles192,
  kMxTiles256,
  kMxPersistent
};

// Cost of a batch in tiles of 64, 128 and 256 rows and columns: rounds over the
// CUs (64: several workgroups follow each other on a CU, so parts of a round)
// times a round's time, given in microseconds at K 4096.
struct TileCost {
  double t64, t128, t256;
};
inline TileCost tile_cost(int M, int N, double us64, double us128, double us256) {
  auto tiles = [&](int b) { return (double)(((int64_t)M + b - 1) / b) * (((int64_t)N + b - 1) / b); };
  const double n64 = tiles(64) / kCUs;
  return TileCost{(n64 < 1 ? 1 : n64) * us64, std::ceil(tiles(128) / kCUs) * us128,
                  std::ceil(tiles(256) / kCUs) * us256};
}

// Of the 32- and 64-row tiles, the ones of 32 rows while they fit the CUs at once,
// or are no more than those of 64 (in us, 32 against 64: 64 x 4096 x 4096 9.1
// against 12.1, 333 x 8192 x 1024 15.4 against 21.5, 32 x 4096 x 14336 9.4 against
// 12.2; 256 x 4096 x 4096 14.0 against 13.2, 64 x 8192 x 28672 50 against 44).
inline MxKernel mx_mid_tiles(int M, int N) {
  const int64_t tiles = (int64_t)((M + 31) / 32) * ((N + 63) / 64);
  return tiles <= kCUs || M <= 32 ? kMxTiles32 : kMxTiles64;
}

// Whether a dense batch is the streamed kernel's: up to 8 rows; up to 16 where the
// 32-row tiles would leave half of the CUs idle (16 rows, streamed against those:
// 4096 -> 4096 7.8 us against 9.0, 8192 -> 1024 12.7 against 14.8, 4096 -> 14336
// 16.6 against 9.6, 8192 -> 28672 45 against 42).
inline bool stream_rows(int M, int N) { return M <= 8 || (M <= 16 && N < 64 * kCUs / 2); }

// Tiles of W rows (8 each) of a workgroup of the streamed kernel for up to 8 rows:
// the widest that still give every CU one.
inline int mx_stream8_tiles(int N) { return N >= 4 * 8 * kCUs ? 4 : N >= 2 * 8 * kCUs ? 2 : 1; }

// bf16 X on an MXFP4 weight, with the LoRA term or without.  Base-only rows of a
// batch with adapters have the base product's bits, so both go by the same rule as
// far as the order of adding up K goes: the streamed kernels', the 32- and 64-row
// tiles', or that of all others.
inline MxKernel mx_weight_kernel_of(int M, int N, bool lora) {
  if (stream_rows(M, N)) return M <= 8 ? kMxStream8 : kMxStream16;
  const TileCost c = tile_cost(M, N, 12.8, 46.5, 85);
  if (c.t64 <= c.t128 && c.t64 <= c.t256) return mx_mid_tiles(M, N);
  if (!lora) return c.t256 <= c.t128 ? kMxPersistent : kMxTiles128;
  // With adapters the shared tiles, whose LoRA term goes through LDS: read from
  // memory into each wave's fragments instead, at the end of the persistent
  // kernel's tiles, it cost 11 us a tile, and the two were level (16943 x 4096 x
  // 14336, 8 slots: 1.69 ms).
  if (c.t128 <= c.t256 * (109. / 85)) return kMxTiles128;
  return large192_tiles(M, N) ? kMxTiles192 : kMxTiles256;
}

// Both operands MXFP4.
inline MxKernel mx_both_kernel_of(int M, int N) {
  const TileCost c = tile_cost(M, N, 6.6, 19.6, 27.5);
  if (c.t64 <= c.t128 && c.t64 <= c.t256) return mx_mid_tiles(M, N);
  return c.t256 <= c.t128 ? kMxPersistent : kMxTiles128;
}

// The experts' products, by the mean rows of an expert (all choices over all
// experts: which experts the batch names, and how often, is not known on the host, so
// each border is that of loads between even ones and a router's with experts twice as
// likely as others).  In us, streamed 8 rows / streamed 16 / 32-row tiles, experts
// equally likely and exp(normal / 2):
//   3 rows: 128 experts, N 2048, K 2048 71 / 74 / 82 and 60 / 58 / 60, K 4096 119 / 151 /
//     142 and 103 / 114 / 103; 64 of 4096 -> 4096 121 / 154 / 149 and 114 / 136 / 127
//   4 rows: 128 experts, N 2048, K 1536 64 / 59 / 73 and 60 / 52 / 60, K 2048 80 / 80 / 88
//     and 76 / 72 / 74, K 2560 90 / 96 / 99 and 82 / 79 / 80, K 4096 136 / 164 / 153 and
//     129 / 146 / 129
//   6 rows, the same: K 1024 58 / 48 / 60 and 61 / 46 / 53, K 1536 71 / 63 / 74 and 75 / 59 /
//     64, K 2048 89 / 85 / 90 and 95 / 81 / 80, K 2560 102 / 103 / 104 and 104 / 94 / 89;
//     32 experts: K 1024 17 / 14 / 17 and 17 / 14 / 16, K 2560 31 / 29 / 28 and 32 / 29 / 28,
//     K 2048, N 8192 89 / 84 / 91 and 94 / 82 / 86
//   8 rows: K 1536 87 / 66 / 74 and 87 / 63 / 66, K 2048 111 / 89 / 92 and 112 / 88 / 81, K
//     4096 195 / 185 / 156 and 197 / 181 / 144
// The more uneven the load the more the tiles gain (128 of 4096 -> 2048, 6 rows,
// exp(2 normal): 130 / 101 / 62), as a streamed expert's weight is read once per 8 or
// 16 of its rows.
//
// The 32-row tiles against the persistent kernel's of 256 x 256: each expert has half a
// tile more than its rows fill, a small one takes 1.6 us and 1.8 per 1024 of K, a CU's
// large one 2 us and 26, and up to two rounds of those count whole, as do a few tiles
// past one (32 experts of 2048 -> 2048, 256 large tiles or a few more: 96 rows 72
// against 58 evenly, 74 against 98 not).  Small / large, evenly and exp(normal / 2):
// 128 of 2048 -> 2048: 64 rows 203 / 218 and 203 / 236, 96 rows 269 / 227 and 271 / 254;
// of 4096 -> 2048: 80 rows 408 / 428 and 419 / 479, 128 rows 594 / 449 and 594 / 527;
// of 1024 -> 2048: 48 rows 111 / 109 and 112 / 116, 80 rows 158 / 116 and 161 / 136;
// 8 of 2048 -> 2048: 160 rows 30 / 48 and 30 / 49.
inline MxKernel mx_experts_kernel_of(int n_choices, int n_experts, int K, int N) {
  const int rows = n_choices / n_experts;
  if (rows <= 3) return kMxStream8;
  if (rows <= (K <= 1536 ? 8 : K <= 2048 ? 5 : 3)) return kMxStream16;
  const double m = (double)n_choices / n_experts, E = n_experts;
  const double small = E * (m / 32 + 0.5) * ((N + 63) / 64) / kCUs * (1.6 + K * 1.76e-3);
  const double rounds = E * (m < 128 ? 1 : m / 256 + 0.5) * ((N + 255) / 256) / kCUs;
  const double large = (rounds <= 2 ? std::ceil(1.05 * rounds) : 1.05 * rounds + 0.3) * (2 + K * 0.0254);
  return small <= large ? kMxTiles32 : kMxPersistent;
}

// Whether the persistent kernels load the scales four words (16 blocks) a row at a
// time: every row's words have to be whole and aligned to that.
inline bool mx_wide_scales(int K, int64_t ldws, int64_t ldxs = 0) {
  return K % 512 == 0 && ldws % 16 == 0 && ldxs % 16 == 0;
}

// The experts' products on bf16 weights (experts_gemm.hip): 32 x 64 tiles whose K goes
// round over a workgroup's waves, 128 x 128, or 256 x 256.
enum ExpertsKernel { kExpertsFew, kExpertsMid, kExpertsLarge };
inline double expert_tiles(int n_choices, int n_experts, int bm, int tiles_n) {
  // every expert in use (at most one a choice) has half a tile more than its rows fill
  const double used = n_choices < n_experts ? n_choices : n_experts, m = n_choices / used / bm + 0.5;
  return used * (m < 1 ? 1 : m) * tiles_n;
}
// The cheapest, a kernel's rounds over the CUs (which hold one workgroup of the first and
// last, two of the other) times a tile's microseconds, of a start and its 64s of K.  In us
// (few / mid / large), few rows on weights that come from memory:
//   1 x 8 choices of 128 experts, 2048 -> 1536: 13.6 / 32 / 48, and the rows' gradient 12.3 /
//     22 / 37; 1 x 2 of 8, 4096 -> 14336: 48 / 70 and 70 / 184
//   4 x 8 of 128, 2048 -> 1536: 42 / 46 and 44 / 37; 64 x 8: 157 / 156 and 171 / 144
//   30 x 4 of 32, 1024 -> 1024: 16.7 / 20.1 and 16.1 / 17.5; 200 x 4: 21 / 20.5 and 22 / 19.4
// and many (uneven ones, mid / large): 128 experts of 2048 -> 1536, 96 rows each 195 / 228 and
//   203 / 210, 160 rows 252 / 246 and 233 / 231, 256 rows 322 / 304 and 310 / 285; 64 of 4096
//   -> 4096, 96 rows 454 / 559 and 471 / 545, 192 rows 688 / 617 and 663 / 597; 8 of 4096 ->
//   14336, 128 rows 247 / 302 and 275 / 334, 256 rows 356 / 334 and 439 / 356.
// (Where memory is what they wait for, the first two are level: the first counts two thirds
// of its own time in a forward product, four fifths in a gradient, whose W it reads in half
// cache lines.)
inline ExpertsKernel experts_kernel_of(int n_choices, int n_experts, int K, int N, bool forward) {
  const double stages = (K + 63) / 64;
  auto rounds = [](double tiles, int at_once) { return tiles <= at_once ? 1.0 : tiles / at_once; };
  const double few = (forward ? 2.7 + 0.21 * stages : 3.3 + 0.26 * stages) *
                     rounds(expert_tiles(n_choices, n_experts, 32, (N + 63) / 64), kCUs);
  const double mid = (4 + 0.85 * stages) *
                     rounds(expert_tiles(n_choices, n_experts, 128, (N + 127) / 128), 2 * kCUs);
  const double large = (6 + 1.3 * stages) *
                       rounds(expert_tiles(n_choices, n_experts, 256, (N + 255) / 256), kCUs);
  return few < mid && few < large ? kExpertsFew : mid <= large ? kExpertsMid : kExpertsLarge;
}

// Their weights' gradients [M][N] (experts_weights.hip): 256 x 256 tiles, or, as long as the
// CUs do not all get one of those, 128 x 128, two workgroups a CU (large / 128, us: 8 experts
// of 64 rows, 1032 x 520, 16 / 13, of 1024 rows 67 / 50; 2 of 256 rows, 1024 x 1024, 18 / 11;
// but 8 of 256, 4096 x 14336, 410 / 493, 128 of 64, 2048 x 1536, 232 / 304).
inline bool experts_weights_large(int M, int N, int n_experts) {
  return (int64_t)((M + 255) / 256) * ((N + 255) / 256) * n_experts > kCUs;
}

}  // namespace lora
