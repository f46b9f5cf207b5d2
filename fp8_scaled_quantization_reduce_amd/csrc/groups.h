// groups.h -- ragged groups of rows (the rows of each expert), shared by the
// grouped quantizer and the grouped GEMMs.
//
// The rows of group e are offsets[e] .. offsets[e + 1] - 1 of a buffer of
// `rows` rows.  The offsets are device data that the host never sees, so a
// launch covers the most tiles that any offsets could need (max_tiles) and
// each block looks its tile up: a wave reads 64 groups at a time, counts
// their tiles and scans the counts.  Offsets are clamped to 0 .. rows and to
// not decrease, so whatever they hold, every tile lies inside the buffer.
//
// The token-contiguous (columnwise) copies give every group whole blocks of
// 128 columns: with tiles of 128 rows, tile t of the numbering below is
// columns 128 t .. 128 t + 127 of such a copy.
#ifndef FP8Q_GROUPS_H
#define FP8Q_GROUPS_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

struct GroupTile {
    int group; // the tile's group
    int row0;  // first row of the group
    int size;  // rows of the group
    int tile;  // tile within the group
};

// Inclusive sums over the wave's lanes.
__device__ __forceinline__ int wave_scan_i32(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// Rows lo .. lo + size - 1 of group g (nothing for g >= groups).
__device__ __forceinline__ void group_rows(const int32_t *offsets, int groups, int rows, int g, int &lo, int &size)
{
    const int a = offsets[min(g, groups)], b = offsets[min(g + 1, groups)];
    lo = min(max(a, 0), rows);
    size = min(max(b, lo), rows) - lo;
}

// The group that holds tile t when every group is cut into tiles of kTile
// rows (a wave-uniform answer; all 64 lanes must call it).  false: there are
// not that many tiles; `tiles` is then their number.
template <int kTile>
__device__ __forceinline__ bool find_tile(const int32_t *offsets, int groups, int rows, int t, GroupTile &gt,
                                          int &tiles)
{
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int g0 = 0; g0 < groups; g0 += 64) {
        int lo, size;
        group_rows(offsets, groups, rows, g0 + lane, lo, size);
        const int count = (int)(((unsigned)size + kTile - 1) / kTile);
        const int sum = wave_scan_i32(count);
        const unsigned long long past = __ballot(base + sum > t);
        if (past) {
            const int l = __ffsll(past) - 1;
            gt.group = g0 + l;
            gt.row0 = __builtin_amdgcn_readlane(lo, l);
            gt.size = __builtin_amdgcn_readlane(size, l);
            gt.tile = t - (base + __builtin_amdgcn_readlane(sum - count, l));
            return true;
        }
        base += __builtin_amdgcn_readlane(sum, 63);
    }
    tiles = base;
    return false;
}

// The most tiles of `tile` rows that `groups` groups over `rows` rows can have.
inline int64_t max_tiles(int64_t rows, int groups, int tile)
{
    return rows / tile + (rows < groups ? rows : groups);
}

} // namespace fp8q

#endif // FP8Q_GROUPS_H
