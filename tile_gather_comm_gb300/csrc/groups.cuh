// groups.cuh -- rows sorted by expert: group e holds rows [offsets[e], offsets[e+1]).
// Every read of the offsets goes through group_range, which keeps whatever they hold inside
// [0, M]: a bad value costs wrong results, never an access outside the tensors.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace tgc {

struct RowRange {
    int begin, end;  // begin <= end, both in [0, M]
};

// offsets == nullptr: one group of all M rows.
__host__ __device__ inline RowRange group_range(const int32_t *offsets, int e, int M) {
    if (offsets == nullptr) return {0, M};
    int a = offsets[e], b = offsets[e + 1];
    a = a < 0 ? 0 : a > M ? M : a;
    b = b < a ? a : b > M ? M : b;
    return {a, b};
}

// Of the n tiles that a group has from place `first` of a list on, how many the list of `listed` tiles
// holds.  Offsets that decrease give groups that overlap, with more tiles in all than the list that M
// rows and the number of groups size; what lies past its end does not exist.
__host__ __device__ inline int listed_tiles(int64_t first, int n, int64_t listed) {
    return first >= listed ? 0 : listed - first < n ? (int)(listed - first) : n;
}

// The place in that list behind n tiles from place `at` on: never past its end, so neither a place nor
// its product with what the list's length was checked against leaves 32 bits (n: the tiles of up to 32
// groups of at least 128 rows a tile).
__host__ __device__ inline int listed_place(int at, int n, int listed) { return at + n < listed ? at + n : listed; }

// Warp-collective: tile `t` of the list that cuts every group into tiles of `tile` rows, in
// order.  Returns the group, or -1 past the last tile; *index is the tile's place inside it.
__device__ __forceinline__ int find_group_tile(const int32_t *offsets, int ngroups, int M, int tile, int t, int lane,
                                               int *index) {
    int base = 0;
    for (int e0 = 0; e0 < ngroups; e0 += 32) {
        int n = 0;
        if (e0 + lane < ngroups) {
            const RowRange r = group_range(offsets, e0 + lane, M);
            n = (r.end - r.begin + tile - 1) / tile;
        }
        int upto = n;  // inclusive sum over the lanes
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, base + upto > t);
        if (hit != 0) {
            const int l = __ffs(hit) - 1;
            *index = t - base - __shfl_sync(0xffffffffu, upto - n, l);
            return e0 + l;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    *index = 0;
    return -1;
}

}  // namespace tgc
