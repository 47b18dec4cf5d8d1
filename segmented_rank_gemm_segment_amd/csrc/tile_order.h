// Which tile a workgroup of the MFMA kernels takes (plain C++ on the host, so that a
// test without a GPU can walk a grid).
#pragma once

#ifdef __HIPCC__
#define LORA_HD __host__ __device__
#else
#define LORA_HD
#endif

namespace lora {

// Tile order of the MFMA kernels.  Workgroup b runs on XCD b % 8 (the
// dispatcher deals consecutive ids round robin over the eight XCDs), and
// each XCD walks its tiles in groups of M-tiles sweeping N, so that
// neighbours share operand tiles in one L2.  Batches of at most
// kHeavyMaxTilesM M-tiles with at least 8 N-tiles: XCD x owns N-tiles
// [x tiles_n / 8, (x + 1) tiles_n / 8) of every M-tile, in groups of 16
// M-tiles (measured 2-4% faster than 8 at 9 M-tiles of 2304 rows), so any
// M-tile's work spreads over all eight XCDs, and an M-tile `heavy` (>= 0)
// comes before the groups, all of its tiles of the XCD first.  Larger batches: XCD x takes
// the x-th eighth of the order over all tiles in groups of 8 M-tiles (each
// XCD then holds a few M-tiles' X rows and streams W, half the L2 misses of
// the N split at 67 M-tiles).  Returns false for a workgroup past its XCD's tiles.
// tile_grid is the launch size that covers every tile.  SPARE: the grid may have more
// workgroups than that, which take none (a comparison that dense batches do without:
// it moved registers in the 256 x 256 kernels, prefill 1787 us to 1809).
constexpr int kTileGroup = 8;
constexpr int kTileGroupSplit = 16;   // M-tiles per group with the N split
constexpr int kHeavyMaxTilesM = 32;
LORA_HD inline bool n_split(int tiles_m, int tiles_n) {
  return tiles_n >= 8 && tiles_m <= kHeavyMaxTilesM;
}
LORA_HD inline int tile_grid(int tiles_m, int tiles_n) {
  return n_split(tiles_m, tiles_n) ? 8 * ((tiles_n + 7) / 8) * tiles_m
                                   : (tiles_m * tiles_n + 7) / 8 * 8;
}
template <bool SPARE>
LORA_HD inline bool tile_order(int b, int tiles_m, int tiles_n, int heavy, int &m_idx,
                               int &n_idx) {
  const int x = b & 7, j = b >> 3;
  int n_lo, nx, t;
  if (n_split(tiles_m, tiles_n)) {
    n_lo = x * tiles_n / 8;
    nx = (x + 1) * tiles_n / 8 - n_lo;
    if (j >= nx * tiles_m) return false;
    t = j;
  } else {
    n_lo = 0;
    nx = tiles_n;
    t = x * ((tiles_m * tiles_n + 7) / 8) + j;
    if (t >= tiles_m * tiles_n) return false;
    if (SPARE && j >= (tiles_m * tiles_n + 7) / 8) return false;   // the next XCD's
  }
  int tm = tiles_m;
  if (heavy >= 0) {
    if (t < nx) {
      m_idx = heavy;
      n_idx = n_lo + t;
      return true;
    }
    t -= nx;
    tm = tiles_m - 1;
  }
  const int G = n_split(tiles_m, tiles_n) ? kTileGroupSplit : kTileGroup;
  const int grp = t / (G * nx);
  const int first_m = grp * G;
  const int gcnt = G < tm - first_m ? G : tm - first_m;
  const int tin = t - grp * G * nx;
  m_idx = first_m + tin % gcnt;
  if (heavy >= 0 && m_idx >= heavy) ++m_idx;
  n_idx = n_lo + tin / gcnt;
  return true;
}

// Workgroups for an experts' product of up to tiles_m M-tiles: they find the
// number there are themselves, and either tile order of it has to fit.
inline int expert_grid(int tiles_m, int tiles_n) {
  const int split = tiles_m < kHeavyMaxTilesM ? tiles_m : kHeavyMaxTilesM;
  const int a = (tiles_m * tiles_n + 7) / 8 * 8, b = 8 * ((tiles_n + 7) / 8) * split;
  return a > b ? a : b;
}
}  // namespace lora
