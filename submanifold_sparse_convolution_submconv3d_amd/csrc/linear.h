// Shared by the grouped matrix products (linear.hip): arguments, and which rows a block's tile is of.
#pragma once

#include "attention.h"

namespace sc {

struct LinearArgs {
    const void *x, *w, *g;  // rows [nx, cin] at x_row, weights [groups, cout, cin], gradient [n, cout] at g_row
    void *out;              // y [n, cout], dx [n, cin] (at out_row), or dw
    const float *bias;      // [groups, cout], or null
    float *db;              // [groups, cout], or null
    const int32_t *off;     // [groups + 1]
    const int32_t *rows;    // row of x of each position, or null for the position itself
    int64_t x_row, g_row, out_row;
    int32_t n, nx;
    int groups, cin, cout;
    // LINEAR_DW in pieces of `chunk` positions of a group (0: whole groups): the sums of piece p, as tiles of
    // `chunk` positions of all parts are counted, stand in part [p][cout][cin] and db_part [p][cout].
    int chunk;
    float *part, *db_part;
};

// Positions [beg, end) of a part: part 0 lies before the first offset, part p of 1..groups is group
// p - 1, part groups + 1 lies behind the last.  Each bound is the largest offset so far, clamped to
// [0, n]: offsets that do not ascend leave groups empty, no position is in two parts and none in
// no part.
struct Part {
    int index, beg, end;
    uint32_t tile;  // of the part
};

__device__ __forceinline__ int lanes_prefix_max(int v)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(v, o, 64);
        if ((int)lane_id() >= o && y > v) v = y;
    }
    return v;
}

// Bound of part index + lane among 64 parts: the end of each; `before`: the end of part index - 1.
__device__ __forceinline__ int part_ends(const LinearArgs &A, int index, int before)
{
    const int p = index + (int)lane_id();
    int o = p <= A.groups ? A.off[p] : (p == A.groups + 1 ? A.n : 0);
    o = o < 0 ? 0 : (o > A.n ? A.n : o);
    if (lane_id() == 0 && before > o) o = before;
    return lanes_prefix_max(o);
}

// The part that tile number t is of, tiles of `size` positions counted part after part without
// gaps.  False past the last.  The same in all lanes; a wave looks at 64 parts at a time.
__device__ __forceinline__ bool find_tile(const LinearArgs &A, int size, uint32_t t, Part *part)
{
    int before = 0;
    uint32_t tiles = 0;
    for (int index = 0; index < A.groups + 2; index += 64) {
        const int end = part_ends(A, index, before);
        int beg = __shfl_up(end, 1, 64);
        if (lane_id() == 0) beg = before;
        const uint32_t own = ((uint32_t)(end - beg) + size - 1) / size;
        uint32_t sum = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t y = __shfl_up(sum, o, 64);
            if ((int)lane_id() >= o) sum += y;
        }
        const uint64_t past = __ballot(tiles + sum > t);
        if (past) {
            const int at = __builtin_ctzll(past);
            part->index = index + at;
            part->beg = __builtin_amdgcn_readlane(beg, at);
            part->end = __builtin_amdgcn_readlane(end, at);
            part->tile = t - (tiles + (uint32_t)__builtin_amdgcn_readlane((int)(sum - own), at));
            return true;
        }
        tiles += (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
        before = __builtin_amdgcn_readlane(end, 63);
    }
    return false;
}

// The pieces of group `group`: the number of its first tile of `size` positions, and how many it has.
__device__ __forceinline__ void group_tiles(const LinearArgs &A, int size, int group, uint32_t *first, uint32_t *count)
{
    int before = 0;
    uint32_t tiles = 0;
    for (int index = 0;; index += 64) {
        const int end = part_ends(A, index, before);
        int beg = __shfl_up(end, 1, 64);
        if (lane_id() == 0) beg = before;
        const uint32_t own = ((uint32_t)(end - beg) + size - 1) / size;
        uint32_t sum = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t y = __shfl_up(sum, o, 64);
            if ((int)lane_id() >= o) sum += y;
        }
        const int at = group + 1 - index;  // the part's lane
        if (at < 64) {
            *count = (uint32_t)__builtin_amdgcn_readlane((int)own, at);
            *first = tiles + (uint32_t)__builtin_amdgcn_readlane((int)sum, at) - *count;
            return;
        }
        tiles += (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
        before = __builtin_amdgcn_readlane(end, 63);
    }
}

// Positions of group `group`.
__device__ __forceinline__ void group_bounds(const LinearArgs &A, int group, Part *part)
{
    int before = 0;
    for (int index = 0;; index += 64) {
        const int end = part_ends(A, index, before);
        const int at = group + 1 - index;  // the part's lane
        if (at < 64) {
            part->index = group + 1;
            part->end = __builtin_amdgcn_readlane(end, at);
            part->beg = at ? __builtin_amdgcn_readlane(end, at - 1) : before;
            part->tile = 0;
            return;
        }
        before = __builtin_amdgcn_readlane(end, 63);
    }
}

// Tiles of `size` positions in all parts, at most.
static inline int64_t most_tiles(int64_t n, int groups, int size) { return n / size + groups + 2; }

enum { LINEAR_Y, LINEAR_DX, LINEAR_DW };

// Tiles of a call in tiles of `size` squared, at most (LINEAR_DW with a chunk: of all pieces).
static inline int64_t linear_tiles(int64_t n, int groups, int cin, int cout, int kind, int chunk, int size)
{
    const int64_t in = (cin + size - 1) / size, out = (cout + size - 1) / size;
    if (kind == LINEAR_DW) return in * out * (chunk ? most_tiles(n, groups, chunk) : groups);
    return most_tiles(n, groups, size) * (kind == LINEAR_Y ? out : in);
}
// Blocks of a call's largest launch; a launch holds 2^24 of them.
int64_t linear_blocks(int64_t n, int groups, int cin, int cout, int dtype, int kind);
int grouped_linear(LinearArgs A, int dtype, int kind, void *workspace, hipStream_t st);
int grouped_linear_big(const LinearArgs &A, int dtype, int kind, int size, hipStream_t st);
size_t linear_dw_workspace(int64_t n, int groups, int cin, int cout, int dtype);

static __device__ __attribute__((aligned(16))) const uint32_t zero_piece[4] = {0, 0, 0, 0};

// A piece of 16 bytes of a row is loaded without a branch, so that loads stay in flight: where the row ends inside it,
// from s elements earlier, which are dropped later.  (Rows have a whole piece or more.)
__device__ __forceinline__ Raw16 drop(Raw16 v, int s, const float *)  // s < 4
{
    if (s & 1) v = Raw16{v[1], v[2], v[3], 0};
    if (s & 2) v = Raw16{v[2], v[3], 0, 0};
    return v;
}
__device__ __forceinline__ Raw16 drop(Raw16 v, int s, const uint16_t *)  // s < 8
{
    if (s & 1) v = Raw16{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    if (s & 2) v = Raw16{v[1], v[2], v[3], 0};
    if (s & 4) v = Raw16{v[2], v[3], 0, 0};
    return v;
}
__device__ __forceinline__ Raw16 load_global(const void *p) { return *(const __attribute__((address_space(1))) Raw16Any *)(uintptr_t)p; }
// Elements of the piece at `at` past the row's `end`, if it has any before it.
template <int V>
__device__ __forceinline__ int past(int at, int end) { return at < end && at + V > end ? at + V - end : 0; }

}  // namespace sc
