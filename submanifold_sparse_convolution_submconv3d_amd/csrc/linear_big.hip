// Grouped matrix products of aligned rows in large tiles (see linear.hip for the products).
//
// Blocks stay on the card and walk tiles of BM x BN: of 256 x 256 (bf16; eight waves, one block a compute unit) or of
// 128 x 128 (both types; four waves, two blocks).  Both sides' tiles are copied straight into a ring of five places in
// LDS, 64 of k in bf16 and 32 in fp32 a step (rows of 128 bytes: copies of 64-byte rows take 0.56 us for 32 KB a compute
// unit, of 128-byte rows 0.34), and on into the next tile, so that a tile's end costs the stores alone.  (Five places of
// one side's step each, 32 KB, let copies run a side further ahead than two of a whole step, in the same LDS.)  In a step,
// each wave multiplies 32x32 blocks on the matrix cores in four quarters of 16 of k; the operands of the next quarter are
// read from LDS meanwhile.  Before the last quarter its operands are in registers: after the step's one barrier there the
// next step's copies, which have landed, are read, and the places that are done with are filled again.
//
// Measured, 8 groups over 40,768 rows of 1024 -> 4096 in bf16 (342 GFLOP a product): forward 347-410 us, dx 330-375,
// dW with db 400-470 (the lower when cool; in a row the card's power holds the clock near 1.8 GHz): 0.73-1.03 PFLOP/s.
// What bounds them then is the matrix cores' waiting for operands: they are busy 67% of the time in dx, 52% in the forward,
// 43% in dW, whose operands come through transposing reads of LDS, two a piece; and dx's 2.56 rounds of tiles take three.
// Tiles of 128 in fp32, 8 x 8192 rows of 1024 -> 1024: 1064, 1041 and 1102 us, 125-132 TFLOP/s of the 152 that a library's
// product of 8192^3 reaches.
#include <type_traits>

#include "linear.h"

namespace sc {

// A tile of the result: rows m0 .. m_end of part, from column n0 on; k_end terms a sum.
struct BigTile {
    int m0, m_end, n0, k_end, group;
    int beg, piece;  // LINEAR_DW: first position of the group or of its piece, and the piece's number
    bool real, any;
};

// The tiles of a call.  Up to 62 groups a lane keeps its part's end and tile numbers.
template <int KIND, int BM, int BN>
struct BigTiles {
    const LinearArgs &A;
    uint32_t m_total, n_tiles, total;
    int end, beg;         // of the lane's part
    uint32_t tiles_end;   // tiles of the parts up to the lane's
    int rank;             // LINEAR_DW: of the lane's group among all, the longest first
    bool kept;
    static constexpr bool DW = KIND == LINEAR_DW;

    __device__ __forceinline__ explicit BigTiles(const LinearArgs &args) : A(args)
    {
        n_tiles = ((KIND == LINEAR_Y ? A.cout : A.cin) + BN - 1) / BN;
        kept = A.groups + 2 <= 64;
        rank = 0;
        const uint32_t m_tiles = DW ? (A.cout + BM - 1) / BM : 1;
        if (DW && !A.chunk) {
            m_total = (uint32_t)A.groups * m_tiles;
            if (kept) {
                part_of(0, 0);
                const int group = (int)lane_id() - 1, len = end - beg;
                for (int g = 0; g < A.groups; ++g) {
                    const int other = __builtin_amdgcn_readlane(len, g + 1);
                    rank += other > len || (other == len && g < group);
                }
                if (group < 0 || group >= A.groups) rank = -1;
            }
        } else {
            m_total = 0;
            int before = 0;
            for (int index = 0; index < A.groups + 2; index += 64) {
                part_of(index, before);
                m_total += (uint32_t)__builtin_amdgcn_readlane((int)tiles_end, 63);
                before = __builtin_amdgcn_readlane(end, 63);
            }
            m_total *= m_tiles;
        }
        total = m_total * n_tiles;
    }
    // The lane's part among 64 from `index` on.
    __device__ __forceinline__ void part_of(int index, int before)
    {
        end = part_ends(A, index, before);
        beg = __shfl_up(end, 1, 64);
        if (lane_id() == 0) beg = before;
        const uint32_t size = DW ? (A.chunk ? A.chunk : 1) : BM;
        tiles_end = ((uint32_t)(end - beg) + size - 1) / size;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t y = __shfl_up(tiles_end, o, 64);
            if ((int)lane_id() >= o) tiles_end += y;
        }
    }
    // Tile number t.  Tiles of GROUP rows of tiles follow each other column by column: the blocks
    // of an XCD, which work on neighbouring numbers, share few rows of either side.
    static constexpr uint32_t GROUP = 8;
    __device__ __forceinline__ BigTile at(uint32_t t)
    {
        BigTile b;
        b.any = t < total;
        b.m0 = b.m_end = b.n0 = b.k_end = b.group = b.beg = b.piece = 0;
        b.real = false;
        if (!b.any) return b;
        const uint32_t g = t / (GROUP * n_tiles), r = t - g * GROUP * n_tiles, rows = m_total - g * GROUP < GROUP ? m_total - g * GROUP : GROUP;
        const uint32_t n = r / rows, m = g * GROUP + (r - n * rows);
        b.n0 = n * BN;
        const uint32_t m_tiles = DW ? (A.cout + BM - 1) / BM : 1, which = m / m_tiles;  // DW: of the groups by length, or of the pieces
        if (DW && !A.chunk) {
            b.m0 = (m - which * m_tiles) * BM;
            b.m_end = A.cout;
            b.real = true;
            if (kept) {
                const int at = __builtin_ctzll(__ballot(rank == (int)which));
                b.group = at - 1;
                b.beg = __builtin_amdgcn_readlane(beg, at);
                b.k_end = __builtin_amdgcn_readlane(end, at) - b.beg;
            } else {
                Part p;
                group_bounds(A, which, &p);
                b.group = which;
                b.beg = p.beg;
                b.k_end = p.end - p.beg;
            }
        } else {
            int index = 0, before = 0;
            uint32_t tiles = 0;
            if (!kept)
                for (;; index += 64) {
                    part_of(index, before);
                    const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)tiles_end, 63);
                    if (tiles + last > which) break;
                    tiles += last;
                    before = __builtin_amdgcn_readlane(end, 63);
                }
            const int at = __builtin_ctzll(__ballot(tiles + tiles_end > which));
            const int pb = __builtin_amdgcn_readlane(beg, at), pe = __builtin_amdgcn_readlane(end, at);
            const uint32_t first = at ? (uint32_t)__builtin_amdgcn_readlane((int)tiles_end, at ? at - 1 : 0) : 0;
            const int part = index + at;
            b.real = part >= 1 && part <= A.groups;
            b.group = b.real ? part - 1 : 0;
            if constexpr (DW) {
                b.m0 = (m - which * m_tiles) * BM;
                b.m_end = A.cout;
                b.beg = pb + (int)(which - tiles - first) * A.chunk;
                b.k_end = !b.real ? 0 : (pe - b.beg < A.chunk ? pe - b.beg : A.chunk);
                b.piece = which;
            } else {
                b.m0 = pb + (int)(which - tiles - first) * BM;
                b.m_end = pe;
                b.k_end = b.real ? (KIND == LINEAR_Y ? A.cin : A.cout) : 0;  // rows of no group become zeros
            }
        }
        return b;
    }
};

template <typename T> constexpr int BIG_K = 128 / (int)sizeof(T);  // of k a step

// A copy of 64 pieces of 16 bytes straight into LDS.  As an instruction of its own, since the compiler
// lets every transposing read wait for all copies that it knows of; the waits are below.  m0 is a register that the
// compiler keeps for itself and takes no notice of in a clobber list, so it is left as it was (8 groups over 40,768 rows of
// 1024 -> 4096 in bf16: 353 -> 355 us).
__device__ __forceinline__ void copy_pieces(const char *from, uint32_t lds)
{
    uint32_t kept;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(kept) : "v"(from), "s"(lds) : "memory");
}

// v[q] of the lanes l, l ^ 8, l ^ 16, l ^ 24, seen as a matrix of lanes (bits 3 and 4 of the lane's number) and q, is
// transposed.
__device__ __forceinline__ void trade_lanes(Raw16 (&v)[4])
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            auto r = __builtin_amdgcn_permlane16_swap(v[q][d], v[q + 2][d], false, false);
            v[q][d] = r[0];
            v[q + 2][d] = r[1];
        }
#pragma unroll
        for (int q = 0; q < 4; q += 2) {  // row_ror:8, into the lanes of one half of 16 each
            const int x = (int)v[q][d], y = (int)v[q + 1][d];
            v[q][d] = (uint32_t)__builtin_amdgcn_update_dpp(x, y, 0x128, 0xf, 0xc, false);
            v[q + 1][d] = (uint32_t)__builtin_amdgcn_update_dpp(y, x, 0x128, 0xf, 0x3, false);
        }
    }
}

// WM x WN waves of MB x NB blocks of 32 x 32.
// LINEAR_DW: SUMS: db too.  PART: pieces of groups, whose sums are kept in fp32 for k_linear_join.
template <typename T, int KIND, int WM, int WN, int MB, int NB, bool SUMS, bool PART>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_linear_big(LinearArgs A)
{
    constexpr bool AKS = KIND == LINEAR_DW, BKS = KIND != LINEAR_Y;
    constexpr int BM = 32 * MB * WM, BN = 32 * NB * WN, WAVES = WM * WN, ES = (int)sizeof(T), V = VEC<T>, BK = BIG_K<T>;
    constexpr int ABYTES = BM * 128, BBYTES = BN * 128;
    constexpr uint32_t ARB = AKS ? BM * ES : 128, BRB = BKS ? BN * ES : 128;  // bytes of a row in LDS
    constexpr int CA = ABYTES / 1024 / WAVES, CB = BBYTES / 1024 / WAVES;  // copies of a wave a step
    static_assert(CA * 1024 * WAVES == ABYTES && CB * 1024 * WAVES == BBYTES, "whole copies");
    static_assert(ABYTES == BBYTES, "one ring for both sides");
    constexpr int RING = 5;
    __shared__ __attribute__((aligned(1024))) char smem[RING * ABYTES];
    const uint32_t lds = (uint32_t)(uintptr_t)(SC_LDS char *)smem;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();

    BigTiles<KIND, BM, BN> tiles(A);
    // Blocks are dealt to the 8 XCDs in turn; those of one take neighbouring tiles, that share an L2:
    // each an eighth of all tiles, or, where tiles are of unequal length (whole groups), of each round.  Every
    // other round of these runs backwards, so that a block with a longer tile gets a shorter one next.
    const uint32_t xcd = blockIdx.x % 8, per = gridDim.x / 8, slot = blockIdx.x / 8, share = (tiles.total + 7) / 8;
    const auto tile_at = [&](uint32_t round) {
        uint32_t t;
        bool there;
        if (KIND == LINEAR_DW && !A.chunk) {
            const uint32_t q = xcd * per + slot;
            t = round * gridDim.x + (round % 2 ? gridDim.x - 1 - q : q);
            there = t < tiles.total;
        } else {
            const uint32_t in = slot + round * per;
            t = share * xcd + in;
            there = in < share && t < tiles.total;
        }
        return tiles.at(there ? t : tiles.total);
    };

    // ---- copies: where a lane's piece of each copy is read next ----
    const char *pa[CA], *pb[CB];
    const auto row_a = [&](int i) { return (int)(((wave * CA + i) * 1024 + lane * 16) / ARB); };  // the copy's row in the tile
    const auto row_b = [&](int i) { return (int)(((wave * CB + i) * 1024 + lane * 16) / BRB); };
    const auto piece_a = [&](int i) { return (int)((((wave * CA + i) * 1024 + lane * 16) % ARB / 16) ^ (AKS && ES == 4 ? 0 : swizzle<ARB>(row_a(i)))); };
    const auto piece_b = [&](int i) { return (int)((((wave * CB + i) * 1024 + lane * 16) % BRB / 16) ^ (BKS && ES == 4 ? 0 : swizzle<BRB>(row_b(i)))); };
    const char *zeros = (const char *)zero_piece;
    int source[KIND == LINEAR_Y ? CA : 1];  // rows of x that the next tile takes
    const auto x_rows = [&](const BigTile &t) {
        if constexpr (KIND == LINEAR_Y) {
#pragma unroll
            for (int i = 0; i < CA; ++i) {
                const int p = t.m0 + row_a(i);
                source[i] = p < t.m_end ? (A.rows ? A.rows[p] : p) : -1;
            }
        }
    };
    const auto column = [](int at, int width) { return at + V <= width ? at : width - V; };  // columns past the end: any that exist
    const auto aim_a = [&](const BigTile &t) {
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            if constexpr (KIND == LINEAR_Y) {
                const bool there = source[i] >= 0 && source[i] < A.nx;
                pa[i] = there ? (const char *)A.x + ((int64_t)source[i] * A.x_row + piece_a(i) * V) * ES : nullptr;
            } else if constexpr (KIND == LINEAR_DX) {
                const int p = t.m0 + row_a(i) < t.m_end ? t.m0 + row_a(i) : t.m_end - 1;
                pa[i] = (const char *)A.g + ((int64_t)p * A.g_row + piece_a(i) * V) * ES;
            } else {
                pa[i] = (const char *)A.g + ((int64_t)(t.beg + row_a(i)) * A.g_row + column(t.m0 + piece_a(i) * V, A.cout)) * ES;
            }
        }
    };
    const auto aim_b = [&](const BigTile &t) {
        const char *w = (const char *)A.w + (int64_t)t.group * A.cout * A.cin * ES;
#pragma unroll
        for (int i = 0; i < CB; ++i) {
            if constexpr (KIND == LINEAR_Y) {
                const int n = t.n0 + row_b(i) < A.cout ? t.n0 + row_b(i) : A.cout - 1;
                pb[i] = w + ((int64_t)n * A.cin + piece_b(i) * V) * ES;
            } else if constexpr (KIND == LINEAR_DX) {
                pb[i] = w + ((int64_t)row_b(i) * A.cin + column(t.n0 + piece_b(i) * V, A.cin)) * ES;
            } else {
                pb[i] = (const char *)A.x + column(t.n0 + piece_b(i) * V, A.cin) * ES;  // and the row, step by step
            }
        }
    };

    BigTile now = tile_at(0);
    if (!now.any) return;
    // What is copied of each side, and from which k on; A's copies run a step ahead of B's.
    BigTile ta = now, tb = now, after;
    uint32_t now_round = 0, b_round = 0, a_round = 1;  // (of `after`)
    int ka = 0, kb = 0;
    x_rows(ta);
    aim_a(ta);
    aim_b(tb);
    after = tile_at(a_round);
    x_rows(after);

    // LINEAR_DW: the rows of x of the step that is copied next.  A wave's copies take consecutive positions, so
    // their rows' numbers are loaded once a wave, during the quarter before the copies: until then no wait for LDS
    // reads, which counts these loads too, comes between.
    constexpr int ROWS = KIND == LINEAR_DW ? (int)(CB * 1024 / BRB) : 1;
    int step_rows[ROWS];
    const auto look_up = [&]() {
        if constexpr (KIND == LINEAR_DW) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int k = kb + (int)wave * ROWS + r, p = tb.beg + k < A.n ? tb.beg + k : A.n - 1;
                step_rows[r] = k < tb.k_end ? (A.rows ? ((const __attribute__((address_space(4))) int32_t *)(uintptr_t)A.rows)[p] : p) : -1;
            }
        }
    };

    uint32_t fill = lds;  // the place that is filled next
    const auto filled = [&]() { fill = fill == lds + (RING - 1) * ABYTES ? lds : fill + ABYTES; };
    const auto copy_a = [&](int i) {
        const char *from = ka + (AKS ? row_a(i) : piece_a(i) * V) < ta.k_end ? pa[i] : zeros;
        if constexpr (KIND == LINEAR_Y) from = pa[i] ? from : zeros;
        copy_pieces(from, __builtin_amdgcn_readfirstlane(fill + (wave * CA + i) * 1024));
    };
    const auto copy_b = [&](int i) {
        const char *from = kb + (BKS ? row_b(i) : piece_b(i) * V) < tb.k_end ? pb[i] : zeros;
        if constexpr (KIND == LINEAR_DW) {
            constexpr int PER = ROWS / CB;  // rows of a copy
            int r = step_rows[i * PER];
#pragma unroll
            for (int q = 1; q < PER; ++q) r = (int)(lane * 16 / BRB) == q ? step_rows[i * PER + q] : r;
            from = r >= 0 && r < A.nx ? pb[i] + (int64_t)r * A.x_row * ES : zeros;
        }
        copy_pieces(from, __builtin_amdgcn_readfirstlane(fill + (wave * CB + i) * 1024));
    };
    // Each side moves on by a step, and to its next tile; past the last one zeros are copied.
    const auto copied_a = [&]() {
        const int64_t d = AKS ? (int64_t)BK * A.g_row * ES : 128;
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            if constexpr (KIND == LINEAR_Y) pa[i] = pa[i] ? pa[i] + d : nullptr;
            else pa[i] += d;
        }
        filled();
        ka += BK;
        if (ka >= ta.k_end && after.any) {
            ta = after;
            ka = 0;
            aim_a(ta);
            ++a_round;
            after = tile_at(a_round);
            x_rows(after);
        }
    };
    const auto copied_b = [&]() {
        if constexpr (KIND != LINEAR_DW) {
            const int64_t d = BKS ? (int64_t)BK * A.cin * ES : 128;
#pragma unroll
            for (int i = 0; i < CB; ++i) pb[i] += d;
        }
        filled();
        kb += BK;
        if (kb >= tb.k_end) {
            const BigTile t = tile_at(b_round + 1);
            if (t.any) {
                tb = t;
                kb = 0;
                ++b_round;
                aim_b(tb);
            }
        }
    };

    // ---- operands ----
    const uint32_t wm = (wave % WM) * (32 * MB), wn = (wave / WM) * (32 * NB);
    struct Operand {  // k next to each other, or fp32: one address; bf16 a row apart: two for each block
        uint32_t at[8];
    } oa, ob, os;
    const auto make = [&](Operand &o, bool ks, uint32_t rb, uint32_t base, uint32_t first, int blocks) {
        const uint32_t a = lane >> 5, g = (lane >> 4) & 1, t = lane & 15;
        if (!ks) {
            o.at[0] = base + piece_at<128>(first + (lane & 31), a);
        } else if (ES == 4) {
            o.at[0] = base + 4 * a * rb + (first + (lane & 31)) * 4;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= blocks) continue;
                    const uint32_t k = 8 * a + 4 * h + t / 4, piece = first / 8 + 4 * i + g * 2 + (t & 3) / 2;
                    o.at[4 * h + i] = base + (rb == 512 ? piece_at<512>(k, piece) : piece_at<256>(k, piece)) + (t & 1) * 8;
                }
        }
    };
    make(oa, AKS, ARB, lds, wm, MB);
    make(ob, BKS, BRB, lds, wn, NB);
    // db: the WN waves that share rows of grad take one of their MB blocks each, read once more
    static_assert(!SUMS || MB == WN, "a block for each wave");
    float sum = 0.0f;
    if constexpr (SUMS) make(os, AKS, ARB, lds, wm + 32 * (wave / WM), 1);
    // 32 bytes of k: quarter j of the place at offset `from`, block i
    const auto read = [&](const Operand &o, bool ks, uint32_t rb, uint32_t from, int j, int i) {
        if (!ks) return lds_read16((o.at[0] ^ (32 * j)) + from + i * (32 * 128));
        if (ES == 4) {
            Raw16 r;
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = *(const SC_LDS uint32_t *)(uintptr_t)(o.at[0] + from + (8 * j + e) * rb + i * 128);
            return r;
        }
        const u32x2 lo = lds_read_tr(o.at[i] + from + j * (16 * rb)), hi = lds_read_tr(o.at[4 + i] + from + j * (16 * rb));
        return Raw16{lo[0], lo[1], hi[0], hi[1]};
    };
    const auto read_a = [&](uint32_t from, int j, int i) { return read(oa, AKS, ARB, from, j, i); };
    const auto read_b = [&](uint32_t from, int j, int i) { return read(ob, BKS, BRB, from, j, i); };

    f32x16 acc[MB][NB];
    Raw16 fa[2][MB], fb[2][NB];
    // The bias of the wave's columns of a tile, one a lane; sums begin with it.
    static_assert(NB == 2, "a column a lane");
    const auto bias_of = [&](const BigTile &t) {
        if (KIND != LINEAR_Y || !A.bias || !t.real) return 0.0f;
        const int e = t.n0 + (int)wn + (int)lane;
        return A.bias[(int64_t)t.group * A.cout + (e < A.cout ? e : A.cout - 1)];
    };
    const auto begin = [&](float bias) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float b = KIND == LINEAR_Y ? __shfl(bias, 32 * n + 8 * (e / 4) + 4 * (int)(lane >> 5) + e % 4, 64) : 0.0f;
#pragma unroll
                for (int m = 0; m < MB; ++m) acc[m][n][e] = b;
            }
        sum = 0.0f;
    };
    uint32_t place_a = 0, place_b = ABYTES;  // offsets of this step's places
    const auto on = [](uint32_t place, int places) { return place + places * ABYTES >= RING * ABYTES ? place + (places - RING) * ABYTES : place + places * ABYTES; };
    // Products of quarter j, with the next quarter's operands read, and copies made, between them.  The
    // order is fixed: each product is followed by its share of the rest.
    const auto quarter = [&](int j, auto copy, int copies) {
        const uint32_t from_a = j == 3 ? on(place_a, 2) : place_a, from_b = j == 3 ? on(place_b, 2) : place_b;
        const int to = (j + 1) & 1, nj = (j + 1) & 3;
        constexpr int READ_STEPS = MB * NB < 4 ? MB * NB : MB * NB / 2, READS = (MB + NB + READ_STEPS - 1) / READ_STEPS;
#pragma unroll
        for (int q = 0; q < MB * NB; ++q) {
            const int m = q / NB, n = q % NB;
            acc[m][n] = mma_pieces<T>(fb[to ^ 1][n], fa[to ^ 1][m], acc[m][n]);
#pragma unroll
            for (int r = q * READS; r < (q + 1) * READS && r < MB + NB; ++r) {
                if (r < NB) fb[to][r] = read_b(from_b, nj, r);
                else fa[to][r - NB] = read_a(from_a, nj, r - NB);
            }
            constexpr int GAP = MB * NB < 8 ? 1 : 2;  // a copy after every product, or every other
            if (q % GAP == GAP - 1 && q / GAP < copies) copy(q / GAP);
            __builtin_amdgcn_sched_barrier(0x6);  // only arithmetic may cross
        }
        if constexpr (SUMS) {  // (the last quarter's with the one before it, while the place is still whole)
#pragma unroll
            for (int q = j; q < 4 && j < 3; q += j == 2 ? 1 : 4) {
                float v[V], t = 0.0f;
                unpack(read(os, AKS, ARB, place_a, q, 0), v, (const T *)nullptr);
#pragma unroll
                for (int i = 0; i < V; i += 2) t += v[i] + v[i + 1];
                sum += t;
            }
        }
    };

    const auto all_a = [&]() {
#pragma unroll
        for (int i = 0; i < CA; ++i) copy_a(i);
        copied_a();
    };
    const auto all_b = [&]() {
        look_up();
#pragma unroll
        for (int i = 0; i < CB; ++i) copy_b(i);
        copied_b();
    };
    // the ring's five places: A and B of step 0, A and B of step 1, and A of step 2 in the loop
    all_a();
    all_b();
    all_a();
    begin(bias_of(now));
    wait_copies_and_barrier<CA>();
    all_b();
#pragma unroll
    for (int i = 0; i < MB; ++i) fa[0][i] = read_a(place_a, 0, i);
#pragma unroll
    for (int i = 0; i < NB; ++i) fb[0][i] = read_b(place_b, 0, i);
    constexpr bool OUT_F32 = PART || ES == 4;
    constexpr int STORES = MB * NB * (OUT_F32 ? 4 : 2), C0 = CA / 2;
    static_assert(CA <= MB * NB && CB <= MB * NB, "room for the copies between the products");
    bool stored = false;  // the last tile's stores may still be in flight
    for (;;) {
        const BigTile next = tile_at(now_round + 1);
        const float next_bias = bias_of(next);  // loaded long before it is needed
        int k = 0;
        do {
            quarter(0, copy_a, C0);
            quarter(1, [&](int i) { copy_a(C0 + i); }, CA - C0);
            copied_a();
            quarter(2, [&](int) { look_up(); }, KIND == LINEAR_DW ? 1 : 0);
            // All of this step's operands are read and both sides' copies for the next have landed.  Loads
            // and stores count in the order of issue: those after B's copies are A's for the step after
            // it, and before these, at a tile's start, the last one's stores (unless some were left out at an edge).
            if (stored) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(CA + STORES) : "memory");
            else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(CA) : "memory");
            stored = false;
            quarter(3, copy_b, CB);
            copied_b();
            place_a = on(place_a, 2);
            place_b = on(place_b, 2);
            k += BK;
        } while (k < now.k_end);
        // a lane has row l % 32 of each block, its elements in the registers
        const int l = lane & 31, a = lane >> 5;
        const int64_t ld = KIND == LINEAR_DW ? A.cin : A.out_row;
        const int n_end = KIND == LINEAR_Y ? A.cout : A.cin;
        typedef typename std::conditional<PART, float, T>::type Out;
        Out *out = PART ? (Out *)A.part : (Out *)A.out;
        if constexpr (KIND == LINEAR_DW) out += (int64_t)(PART ? now.piece : now.group) * A.cout * A.cin;
        if constexpr (SUMS) {
            sum += other_half(sum);
            const int row = now.m0 + (int)wm + 32 * (int)(wave / WM) + l;
            if (now.n0 == 0 && a == 0 && row < now.m_end) (PART ? A.db_part : A.db)[(int64_t)(PART ? now.piece : now.group) * A.cout + row] = sum;
        }
        // Stores of whole lines: the 16-byte pieces of a row that its two lanes hold are traded among the lanes
        // 8 apart, so that eight lanes have 128 bytes of a row, and a store writes eight rows.
        const bool whole = now.m0 + BM <= now.m_end && now.n0 + BN <= n_end;
        const int j = l / 8;
        const auto put = [&](Raw16 (&v)[4], int m, int first) {  // pieces 2q + a of the 8 from column `first` on
            trade_lanes(v);
            const int e = first + (2 * j + a) * (16 / (int)sizeof(Out)), row = now.m0 + (int)wm + 32 * m + l % 8;
            Out *to = out + (int64_t)row * ld + e;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (whole) *(Raw16Any *)(to + (int64_t)(8 * q) * ld) = v[q];
                else if (row + 8 * q < now.m_end && e < n_end)
                    store_raw(to + (int64_t)(8 * q) * ld, v[q], n_end - e < 16 / (int)sizeof(Out) ? n_end - e : 16 / (int)sizeof(Out));
            }
        };
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            Raw16 v[4];
            if constexpr (OUT_F32) {
#pragma unroll
                for (int n = 0; n < NB; ++n) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[q] = Raw16{__float_as_uint(acc[m][n][4 * q]), __float_as_uint(acc[m][n][4 * q + 1]), __float_as_uint(acc[m][n][4 * q + 2]),
                                     __float_as_uint(acc[m][n][4 * q + 3])};
                    put(v, m, now.n0 + (int)wn + 32 * n);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {  // registers 8h .. + 3 and 8h + 4 .. + 7: 8 elements in a row after the halves' exchange
                    const int n = q / 2, h = q % 2;
                    float t[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[m][n][8 * h + i]), __float_as_uint(acc[m][n][8 * h + 4 + i]), false, false);
                        t[i] = __uint_as_float(r[0]);
                        t[4 + i] = __uint_as_float(r[1]);
                    }
                    v[q] = repack(t, (const uint16_t *)nullptr);
                }
                put(v, m, now.n0 + (int)wn);
            }
        }
        stored = whole;
        ++now_round;
        now = next;
        if (!now.any) break;
        begin(next_bias);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy may land in LDS that the next block owns
}

// Tiles of 256 x 256 in eight waves, a block a compute unit, or of 128 x 128 in four, two blocks.
int grouped_linear_big(const LinearArgs &A, int dtype, int kind, int size, hipStream_t st)
{
    const int64_t tiles = (linear_tiles(A.n, A.groups, A.cin, A.cout, kind, A.chunk, size) + 7) / 8 * 8, most = UNITS * (size == 256 ? 1 : 2);
    const dim3 grid((unsigned)(tiles < most ? tiles : most));
#define LARGE(T, KIND, SUMS, PART) hipLaunchKernelGGL((k_linear_big<T, KIND, 2, 4, 4, 2, SUMS, PART>), grid, dim3(512), 0, st, A)
#define SMALL(T, KIND, SUMS, PART) hipLaunchKernelGGL((k_linear_big<T, KIND, 2, 2, 2, 2, SUMS, PART>), grid, dim3(256), 0, st, A)
#define DW(GO, T)                                                                                              \
    if (A.chunk) { if (A.db) GO(T, LINEAR_DW, true, true); else GO(T, LINEAR_DW, false, true); }               \
    else { if (A.db) GO(T, LINEAR_DW, true, false); else GO(T, LINEAR_DW, false, false); }
    if (dtype == SUBMCONV_F32) {  // 128 throughout: a tile of 256 takes 226 us for 1024 of k
        if (kind == LINEAR_Y) SMALL(float, LINEAR_Y, false, false);
        else if (kind == LINEAR_DX) SMALL(float, LINEAR_DX, false, false);
        else { DW(SMALL, float) }
    } else if (kind == LINEAR_DW) {
        DW(LARGE, uint16_t)
    } else if (size == 256) {
        if (kind == LINEAR_Y) LARGE(uint16_t, LINEAR_Y, false, false);
        else LARGE(uint16_t, LINEAR_DX, false, false);
    } else {
        if (kind == LINEAR_Y) SMALL(uint16_t, LINEAR_Y, false, false);
        else SMALL(uint16_t, LINEAR_DX, false, false);
    }
#undef DW
#undef SMALL
#undef LARGE
    SC_LAUNCHED("grouped_linear");
    return SUBMCONV_OK;
}

}  // namespace sc
