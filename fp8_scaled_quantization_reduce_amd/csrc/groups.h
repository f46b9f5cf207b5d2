// groups.h -- ragged groups of rows (the rows of each expert), shared by the
// grouped quantizer and the grouped GEMMs.
//
// The rows of group e are offsets[e] .. offsets[e + 1] - 1 of a buffer of
// `rows` rows.  The offsets are device data that the host never sees, so a
// launch covers the most tiles that any offsets could need (max_tiles) and
// each block looks its tile up: a wave reads 64 groups at a time, counts
// their tiles and scans the counts (GroupTiles).  Offsets are clamped to 0 .. rows
// and a group that would end before it starts is empty, so whatever they hold,
// every tile lies inside the buffer.  Groups of offsets that decrease may share
// rows, and their tiles then be more than a launch covers (or than 32 bits hold):
// the count of tiles ends at what the groups of one buffer can have.
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

// The groups cut into tiles of kTile rows.  A wave holds 64 groups at a time;
// with at most 64 the offsets are read once.  All 64 lanes must construct it
// and call find, whose answers are wave-uniform.
template <int kTile> struct GroupTiles {
    const int32_t *offsets;
    int groups, rows;
    int lo, size, count, sum; // of group 64 i + lane, for the chunk held
    int total;                // tiles of all groups, at most rows / kTile + groups

    __device__ __forceinline__ void hold(int g0)
    {
        group_rows(offsets, groups, rows, g0 + (threadIdx.x & 63), lo, size);
        count = (int)(((unsigned)size + kTile - 1) / kTile);
        sum = wave_scan_i32(count);
    }
    __device__ __forceinline__ GroupTiles(const int32_t *o, int g, int r) : offsets(o), groups(g), rows(r), total(0)
    {
        for (int g0 = 0; g0 < groups; g0 += 64) {
            hold(g0);
            total = min(total + __builtin_amdgcn_readlane(sum, 63), rows / kTile + groups);
        }
    }
    // the group that holds tile t, 0 <= t < total
    __device__ __forceinline__ GroupTile find(int t)
    {
        int base = 0;
        for (int g0 = 0;; g0 += 64) {
            if (groups > 64) hold(g0);
            const int tiles = __builtin_amdgcn_readlane(sum, 63);
            if (t < base + tiles || g0 + 64 >= groups) {
                const unsigned long long past = __ballot(base + sum > t);
                const int l = past ? __ffsll(past) - 1 : 63;
                const int first = base + __builtin_amdgcn_readlane(sum - count, l);
                return GroupTile{g0 + l, __builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(size, l),
                                 t - first};
            }
            base += tiles;
        }
    }
};

// The most tiles of `tile` rows that `groups` groups over `rows` rows can
// have: sum ceil(m / tile) over at most min(groups, rows) groups with rows.
inline int64_t max_tiles(int64_t rows, int groups, int tile)
{
    return (rows + (rows < groups ? rows : groups) * (tile - 1)) / tile;
}

} // namespace fp8q

#endif // FP8Q_GROUPS_H
