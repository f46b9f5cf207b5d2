// gated_tiles.h -- which tiles a gated product runs in, shared by its launchers
// and the entry points, which tell the caller the workspace.
#ifndef FP8Q_GATED_TILES_H
#define FP8Q_GATED_TILES_H

#include "fp8q_launch.h"
#include "gemm_kernels.h"
#include "groups.h"

namespace fp8q {

enum GatedTile { kGated16, kGatedMid, kGatedPP };

// Slices whose scales the 64-row tiles hold in LDS: K to 14336, the longest
// contraction they were timed at.  Beside their stages there is room for 128.
constexpr int kMidSlices = 112;

// Rows past which a call that writes codes takes no 16-row tiles, so that the
// workspace they need has a bound.
constexpr int64_t kFewRows = 4096;

inline int64_t gated_pp_blocks(int64_t rows, int groups, int64_t F, int cus)
{
    return max_tiles(rows, groups, 256) * (F / 128) + kXcds * (1 + cus / 2);
}

// The tile of a gated product.  Up to 8 rows a group on average the 16-row tiles
// read the weights once, in the smallest pieces.  Above, the tiles whose rounds of a
// block per CU take least, with these times of a round in us (k = K / 4096), from
// one matrix of 512 to 14336 columns, 1 to 1024 rows and K 1024 to 4096, its weights
// in the last-level cache:
//   16 rows x 16   7.6 k, 7 + 3 k at the least, and 3 for the finishing pass of codes
//   64 x 128       4 + 17 k
//   256 x 128      6.5 + 29.5 k (most of them 128 x 128: 6.5 + 26 k)
// 301 rows of 4096 x 4096 take 126, 24.9 and 34.6 us in the three, 32 rows 20, 22.6
// and 32.5, 1024 rows 404, 50 and 38; 32 rows of each of 64 matrices of 1408 x 2048 172, 73
// and 76 (the bytes of the weights: 71).  Past K 4096 the three were not compared: 64
// rows of 4096 columns take 39.5 us in the 64-row tiles at K 8192 and 65 at 14336 (38
// and 63.5 here).  Weights that come from memory add a fifth to a half, most to few
// blocks: the same 64 rows 29 us at K 4096, 55 at 8192, 97 at 14336, and 126 in the
// large tiles at 16384.  Ragged groups count as the worst split of their rows.
inline GatedTile gated_tile(int64_t rows, int groups, int64_t F, int64_t K, bool codes, int cus_)
{
    const int64_t cus = cus_ > 0 ? cus_ : 256, live = rows < groups ? rows : groups;
    auto blocks = [&](int tm, int tn) { return max_tiles(rows, groups, tm) * (F / tn); };
    auto rounds = [&](int tm, int tn) { return (double)((blocks(tm, tn) + cus - 1) / cus); };
    const bool fit16 = !(codes && rows > kFewRows) && blocks(16, 16) <= max_blocks(1024);
    const bool fit64 = K <= kMidSlices * kBK && blocks(64, 128) + kXcds <= max_blocks(kBSThreads);
    if (rows <= 8 * live && fit16) return kGated16;
    const double k = (double)K / 4096.0, all = 7.6 * k * rounds(16, 16), least = 7.0 + 3.0 * k;
    const double t16 = (all > least ? all : least) + (codes ? 3.0 : 0.0), t64 = (4.0 + 17.0 * k) * rounds(64, 128);
    const double pp = (6.5 + (rows <= 128 * live ? 26.0 : 29.5) * k) * rounds(256, 128);
    if (fit64 && t64 < pp) return fit16 && t16 < t64 ? kGated16 : kGatedMid;
    return fit16 && t16 < pp ? kGated16 : kGatedPP;
}

} // namespace fp8q

#endif // FP8Q_GATED_TILES_H
