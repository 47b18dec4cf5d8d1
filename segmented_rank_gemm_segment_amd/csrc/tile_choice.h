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
// experts: which experts the batch names, and how often, is not known on the host).
// `many`: more tiles of 32 x 64 than two rounds of two workgroups to a CU, which
// those tiles need to follow each other without a gap, while the streamed kernels
// have fewer bytes of X for each of W to fetch.  In us, streamed 8 rows / streamed 16 /
// 32-row tiles, one size varied at a time:
//   K, 128 experts, N 2048, 6 rows: 1024 61 / 46 / 66, 2560 104 / 94 / 109, 3584 138 /
//     139 / 146, 4096 163 / 164 / 174; 4 rows 52 / 42 / 64 to 129 / 145 / 160; 8 rows
//     71 / 50 / 69 to 196 / 180 / 178
//   N, 32 experts, K 2048, 6 rows: 1024 16 / 15 / 13, 2048 28 / 25 / 24, 4096 50 / 44 /
//     46, 8192 93 / 82 / 85; 8 rows 18 / 19 / 13 to 110 / 94 / 90
//   experts, K and N 2048, 6 rows: 8 11 / 10 / 9, 48 39 / 35 / 42, 64 52 / 46 / 53, 128
//     94 / 80 / 101; K and N 4096: 16 47 / 47 / 41, 64 167 / 173 / 169
//   up to 3 rows streaming 8 is within 4% of the best on all of these, 10 rows and
//   more in tiles on all but short K with many tiles (64 of K and N 2048 55 against 60)
// The tiles against the 256-tiles, 64 experts of 2048 -> 1536 and 16 of 4096 -> 4096:
// 64 rows 89 against 98 and 80 against 97, 96 rows 116 against 100 and 105 against 99.
inline MxKernel mx_experts_kernel_of(int n_choices, int n_experts, int K, int N) {
  const int rows = n_choices / n_experts;
  const bool many = (int64_t)n_experts * ((N + 63) / 64) > 4 * kCUs;
  if (many && K <= 2560 && rows >= 4 && rows <= 8) return kMxStream16;
  if (rows <= (many ? 6 : 4)) return kMxStream8;
  return rows < 80 ? kMxTiles32 : kMxPersistent;
}

// Whether the persistent kernels load the scales four words (16 blocks) a row at a
// time: every row's words have to be whole and aligned to that.
inline bool mx_wide_scales(int K, int64_t ldws, int64_t ldxs = 0) {
  return K % 512 == 0 && ldws % 16 == 0 && ldxs % 16 == 0;
}

}  // namespace lora
