// fp4q_groups.h -- rows in groups that the device alone knows (fp4q_grouped.hip,
// fp4q_fp8_quantize.hip): group e of `groups` owns rows offsets[e] .. offsets[e + 1] - 1, and a
// workgroup finds the group of its tile by adding up the groups' tiles, 64 at a time, one a lane.
// Device code only; each including file gets its own copy.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {
namespace {

// Offsets outside 0 .. rows are taken as the nearest inside, a group that ends before it starts
// as empty: no group holds a row that does not exist.  (Offsets out of order can make groups that
// overlap, and more tiles than a launch has workgroups for: those are left out.  At most 2^28 rows,
// so that the tiles of 512 such groups are counted in 32 bits.)  With `rest`, the rows of no
// group are two more: those behind the last group, and those before the first.
struct Groups {
    const int* offsets;
    int count;   // groups
    int rows;
    bool rest;

    __device__ __forceinline__ int total() const { return count + (rest ? 2 : 0); }
    __device__ __forceinline__ int bound(int e) const { return min(max(offsets[e], 0), rows); }
    __device__ __forceinline__ void range(int e, int& lo, int& hi) const {
        lo = hi = rows;
        if (e < count) {
            lo = bound(e);
            hi = min(max(offsets[e + 1], lo), rows);
        } else if (e < total()) {
            lo = bound(count);
            if (e > count) hi = min(bound(0), lo), lo = 0;
        }
    }
};

// Sum over the lanes up to and including this one.
__device__ __forceinline__ int wave_sums(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return v;
}

struct GroupTile {
    int group;       // of the tile; -1: past the last tile
    int row, end;    // its first row, and its group's end
    int before;      // tiles of the groups before it
};

// The tiles of `side` rows that the groups take together.
__device__ __forceinline__ int group_tiles(const Groups& g, int side) {
    const int lane = threadIdx.x % 64;
    int tiles = 0;
    for (int c = 0; c < g.total(); c += 64) {
        int lo, hi;
        g.range(c + lane, lo, hi);
        tiles += __builtin_amdgcn_readlane(wave_sums((hi - lo + side - 1) / side), 63);
    }
    return tiles;
}

// Tile `tile` (the same in all lanes).
__device__ __forceinline__ GroupTile group_tile(const Groups& g, int side, int tile) {
    const int lane = threadIdx.x % 64;
    int before = 0;
    for (int c = 0; c < g.total(); c += 64) {
        int lo, hi;
        g.range(c + lane, lo, hi);
        const int mine = (hi - lo + side - 1) / side, sums = wave_sums(mine);
        const uint64_t past = __builtin_amdgcn_ballot_w64(before + sums > tile);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int first = before + __builtin_amdgcn_readlane(sums - mine, l);
            return {c + l, __builtin_amdgcn_readlane(lo, l) + (tile - first) * side, __builtin_amdgcn_readlane(hi, l), first};
        }
        before += __builtin_amdgcn_readlane(sums, 63);
    }
    return {-1, 0, 0, before};
}

// The group number `n` of those that hold a row, in `tile` order with side = rows: tile 0 of it.
__device__ __forceinline__ GroupTile nonempty_group(const Groups& g, int n) {
    const int lane = threadIdx.x % 64;
    for (int c = 0; c < g.total(); c += 64) {
        int lo, hi;
        g.range(c + lane, lo, hi);
        uint64_t some = __builtin_amdgcn_ballot_w64(hi > lo);
        const int here = __builtin_popcountll(some);
        if (n < here) {
            for (; n > 0; --n) some &= some - 1;
            const int l = __builtin_ctzll(some);
            return {c + l, __builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(hi, l), 0};
        }
        n -= here;
    }
    return {-1, 0, 0, 0};
}

}  // namespace
}  // namespace fp4q
