// Shared by the attention kernels (attention.hip, attention_bwd.hip): the ragged tile
// lookup, tiles in LDS, and the matrix products on them.
//
// All products are 32x32 blocks on the matrix cores.  With l = lane, a = l / 32, an
// operand of a product over the head dimension is row l % 32 of a tile, 16 bytes at a time: half a
// holds pieces 2j + a.  (For fp32 that orders the dimension differently from the
// instruction's own order, the same way on both sides, so the sum is the same.)  The
// result block has column l % 32 and rows 8 (i / 4) + 4 a + i % 4 in its 16 registers i.
//
// The kernels always put the rows they own (queries, or keys) in the columns.  A lane
// then owns one query (or key), softmax statistics need one exchange between halves,
// and the result registers, rounded to the operand type, are the second operand of the
// next product, over the other side's rows: its first operand, the transposed tile, is
// read from LDS in the row order those registers have.
#pragma once

#include "rowvec.h"

namespace sc {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

#define SC_LDS __attribute__((address_space(3)))

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// --------------------------------------------------------------------------
// ragged batches
// --------------------------------------------------------------------------

// The rows of a packed ragged batch: entry e has rows [off[e], off[e + 1]).  Seen as
// entries + 2 parts: what lies before the first and after the last offset are parts
// without a counterpart on the other side.  Bounds are clamped to [0, n], so offsets
// that do not ascend cannot lead outside the tensors.
struct Ragged {
    const int32_t *off;
    int entries;
    int64_t n;
    int mult;  // query rows of a token (heads that share a key head), 1 for keys

    __device__ __forceinline__ int64_t bound(int part) const
    {
        if (part <= 0) return 0;
        if (part > entries + 1) return n;
        const int64_t o = off[part - 1];
        return o < 0 ? 0 : (o > n ? n : o);
    }
    // First tile number of a part: tiles of `rows` rows, numbered with gaps so that the
    // number needs the part's own bound alone.
    __device__ __forceinline__ int64_t first_tile(int part, int rows) const { return bound(part) * mult / rows + part; }
};

static inline int64_t ragged_tiles(int64_t n, int entries, int mult, int rows) { return n * mult / rows + entries + 2; }

// A block's share: tile `tile` of a part's rows on its own side, for `which` of the heads (and
// tiles of the other side); where the part lies on both sides, in rows.  `real`: the part is
// an entry.
struct Work {
    uint32_t which;
    bool real;
    int64_t tile, own_beg, own_len, other_beg, other_len;
    // Cut tiles: the block takes piece `piece` of `pieces` of the other side; its partial
    // results have number `index`.
    uint32_t piece, pieces, index;
};

// Tiles that do not fill the card's `slots` blocks another time are cut along the other side,
// so that their pieces do: 1.6 rounds of tiles take the time of 1.6 to 1.7, not of 2.  The
// number of pieces is the one that ends soonest; a larger one has to gain a fifth (partial
// results cost memory traffic).
// slots = 0: nothing is cut.
constexpr uint32_t MAX_PIECES = 5;
__device__ __forceinline__ uint32_t cut_pieces(uint32_t rest, uint32_t slots)
{
    uint32_t best = 1, rounds = 1;
    for (uint32_t n = 2; n <= MAX_PIECES && rest * n <= 2 * slots; ++n) {
        const uint32_t r = (rest * n + slots - 1) / slots;
        if (r * best * 10 < rounds * n * 8) {
            best = n;
            rounds = r;
        }
    }
    return best;
}

// What work number w is: work is all tiles of all parts, `many` times over.  False past the
// end.  The same in all lanes.
//   Up to 254 entries each lane counts the tiles of its EACH parts and a sum over lanes numbers
//   them without gaps, so that the blocks with work spread evenly over the card whatever
//   the lengths, and the bounds come with one memory latency; with more entries tiles are
//   numbered as first_tile has it, and 64 bounds are compared at a time.
constexpr int EACH = 4;
__device__ __forceinline__ bool find_work(const Ragged &own, const Ragged &other, int rows, uint32_t w, uint32_t many, uint32_t slots, bool join, Work *k)
{
    const int parts = own.entries + 2, lane = (int)lane_id();
    int part;
    k->piece = k->index = 0;
    k->pieces = 1;
    if (parts <= 64 * EACH) {
        const int each = (parts + 63) / 64, p0 = lane * each;
        int64_t b[EACH + 1], ob[EACH + 1];
#pragma unroll
        for (int i = 0; i <= EACH; ++i) {
            const int p = p0 + (i < each ? i : each);
            b[i] = own.bound(p < parts ? p : parts);
            ob[i] = other.bound(p < parts ? p : parts);
        }
        uint32_t tiles[EACH], count = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int64_t len = (b[i + 1] - b[i]) * own.mult;  // 0 past the lane's parts
            tiles[i] = len > 0 ? (uint32_t)((len + rows - 1) / rows) : 0;
            count += tiles[i];
        }
        uint32_t sum = count;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t y = __shfl_up(sum, o, 64);
            if (lane >= o) sum += y;
        }
        const uint32_t total = __builtin_amdgcn_readlane(sum, 63);
        if (total == 0) return false;
        const uint32_t all = total * many;
        if (slots) {
            const uint32_t rest = all % slots, full = all - rest, n = cut_pieces(rest, slots);
            if (join) {  // w counts cut tiles
                if (n == 1 || w >= rest) return false;
                k->pieces = n;
                k->index = w * n;
                w += full;
            } else if (n > 1 && w >= full) {
                k->index = w - full;
                if (k->index >= rest * n) return false;
                k->pieces = n;
                k->piece = k->index % n;
                w = full + k->index / n;
            }
        }
        if (w >= all) return false;
        k->which = w / total;
        const uint32_t slot = w - k->which * total;
        const int at = __builtin_ctzll(__ballot(sum > slot));
        uint32_t tile = slot - (sum - count);  // meant in lane `at`
        int64_t beg = b[0], end = b[1], obeg = ob[0], oend = ob[1];
        part = p0;
#pragma unroll
        for (int i = 1; i < EACH; ++i)  // which of the lane's parts
            if (part == p0 + i - 1 && tile >= tiles[i - 1]) {
                tile -= tiles[i - 1];
                part = p0 + i;
                beg = b[i];
                end = b[i + 1];
                obeg = ob[i];
                oend = ob[i + 1];
            }
        part = __builtin_amdgcn_readlane(part, at);
        k->tile = (uint32_t)__builtin_amdgcn_readlane(tile, at);
        k->own_beg = __builtin_amdgcn_readlane((int)beg, at);
        k->own_len = __builtin_amdgcn_readlane((int)end, at) - k->own_beg;
        k->other_beg = __builtin_amdgcn_readlane((int)obeg, at);
        k->other_len = __builtin_amdgcn_readlane((int)oend, at) - k->other_beg;
    } else {
        const uint32_t numbers = (uint32_t)(own.n * own.mult / rows + own.entries + 2);
        k->which = w / numbers;
        if (join || k->which >= many) return false;
        const uint32_t slot = w - k->which * numbers;
        int lo = 0, hi = parts;
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) / 64;
            const int p = lo + lane * step;
            const uint64_t le = __ballot(p < hi && own.first_tile(p, rows) <= slot);
            const int count = ~le ? __builtin_ctzll(~le) : 64;
            const int next = lo + (count > 1 ? count - 1 : 0) * step;
            hi = next + step < hi ? next + step : hi;
            lo = next;
        }
        part = __builtin_amdgcn_readfirstlane(lo);
        k->tile = slot - own.first_tile(part, rows);
        k->own_beg = own.bound(part);
        k->own_len = own.bound(part + 1) - k->own_beg;
        k->other_beg = other.bound(part);
        k->other_len = other.bound(part + 1) - k->other_beg;
    }
    if (k->own_len < 0) k->own_len = 0;
    k->real = part >= 1 && part <= own.entries;
    if (!k->real || k->other_len < 0) k->other_len = 0;
    return true;
}

// The part that holds a row (mult = 1).
__device__ __forceinline__ int find_part(const Ragged &r, int64_t row)
{
    int lo = 0, hi = r.entries + 2;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const int p = lo + (int)lane_id() * step;
        const uint64_t le = __ballot(p < hi && r.bound(p) <= row);
        const int count = ~le ? __builtin_ctzll(~le) : 64;
        const int next = lo + (count > 1 ? count - 1 : 0) * step;
        hi = next + step < hi ? next + step : hi;
        lo = next;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Work number of a block: runs of 4 go to one XCD (blocks are dealt to the 8 XCDs in
// turn), so that neighbours, which read the same keys, share an L2.  Grids are whole
// multiples of 32; numbers past the work are idle.
constexpr int XCD_RUN = 4;
static inline unsigned xcd_grid(int64_t total) { return (unsigned)((total + 8 * XCD_RUN - 1) / (8 * XCD_RUN) * (8 * XCD_RUN)); }
__device__ __forceinline__ unsigned xcd_work()
{
    const unsigned b = blockIdx.x, g = b / (8 * XCD_RUN), in = b % (8 * XCD_RUN);
    return g * (8 * XCD_RUN) + (in % 8) * XCD_RUN + in / 8;
}

// [n, heads, dim] in device memory: element (i, h, d) at i * row + h * head + d.
struct Heads {
    const void *p;
    int64_t row, head;
};

// --------------------------------------------------------------------------
// tiles in LDS
// --------------------------------------------------------------------------

// A tile is rows of RB bytes (the padded head).  16-byte pieces of row r are permuted by
// an exclusive or with swizzle(r): 16 rows read at one piece (the operand over the head
// dimension), and 4 rows read at four neighbouring pieces (the transposed operand), then fall on
// different banks for every RB.
template <int RB>
__device__ __forceinline__ uint32_t swizzle(uint32_t row)
{
    uint32_t s = (row >> 2) & 3;
    if (RB % 256 == 0) s |= (row & 3) << 2;
    else if (RB % 128 == 0) s |= ((row >> 1) & 1) << 2;
    return s;
}

template <int RB>
__device__ __forceinline__ uint32_t piece_at(uint32_t row, uint32_t piece)
{
    return row * RB + ((piece ^ swizzle<RB>(row)) << 4);
}

__device__ __forceinline__ Raw16 lds_read16(uint32_t at) { return *(const SC_LDS Raw16 *)(uintptr_t)at; }
__device__ __forceinline__ void lds_write16(uint32_t at, Raw16 v) { *(SC_LDS Raw16 *)(uintptr_t)at = v; }

// Waits until at most N of this wave's vector-memory loads are in flight, and all its LDS
// accesses are done; then a barrier.  Copies into LDS count as loads and the compiler
// does not wait for them by itself.
template <int N>
__device__ __forceinline__ void wait_copies_and_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Tiles of 32 rows of two tensors, copied one after the other into rings of RING places in
// LDS, 64 pieces of 16 bytes (1 KB) a copy.  The first half of a block's waves copies the
// one tensor, the second half the other, so a wave has one pointer to move.  Rows past the
// tensor's part and pieces past dim become zeros.
//   DIRECT: straight into LDS through bounds-checked buffer copies, which stay in flight.
//   Needs 16-byte alignment, and rows that do not overlap (the check is on the offset).
//   Otherwise: loads and LDS writes, any alignment and row distance.
constexpr uint32_t OUT_OF_RANGE = 0x80000000u;

// A buffer of `bytes` from p on.  Both are the same in all lanes; said so explicitly, since a
// copy whose buffer the compiler holds in vector registers is put into a loop over lanes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scalar_rsrc(const void *p, int bytes)
{
    const uint64_t u = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    const uint64_t q = (uint64_t)hi << 32 | lo;  // (the builtin returns a signed int)
    return __builtin_amdgcn_make_buffer_rsrc((void *)q, (short)0, __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

template <typename T, int RB, int WAVES, int RING, bool DIRECT>
struct Fill {
    static constexpr int TILE = 32 * RB, PER = RB / 16 / WAVES;  // copies of a wave for a tile
    static_assert(RB / 16 % WAVES == 0 && WAVES % 2 == 0, "whole copies, waves of one tensor");
    uint32_t off[PER];      // byte offset of the lane's piece from row 0 of a tile
    uint32_t to;            // LDS address of the wave's first copy in place 0
    int64_t row_bytes;      // of the wave's tensor
    bool second;            // which one it is
    const char *ptr;        // row 0 of the next tile
    int left;               // its rows that exist (more than 32: all do)
    uint32_t place;         // its place's offset in the ring

    // lds_a, lds_b: the rings; row_a, row_b: distances between rows in elements (both 0 for
    // next_grouped).
    __device__ __forceinline__ void init(uint32_t lds_a, uint32_t lds_b, int64_t row_a, int64_t row_b, int dim)
    {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
        second = wave >= WAVES / 2;
        const uint32_t first = (wave - (second ? WAVES / 2 : 0)) * PER * 1024;
        to = (second ? lds_b : lds_a) + first;
        row_bytes = (second ? row_b : row_a) * (int64_t)sizeof(T);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t in = first + i * 1024 + lane * 16, r = in / RB, piece = (in % RB / 16) ^ swizzle<RB>(r);
            off[i] = piece * VEC<T> < (uint32_t)dim ? r * (uint32_t)row_bytes + piece * 16 : OUT_OF_RANGE;
        }
    }
    // The next tile is the first: `rows` rows from a and b on.
    __device__ __forceinline__ void start(const T *a, const T *b, int rows)
    {
        ptr = (const char *)(second ? b : a);
        left = rows;
        place = 0;
    }
    __device__ __forceinline__ void next()
    {
        const int n = left < 0 ? 0 : (left > 32 ? 32 : left);
        if constexpr (DIRECT) {
            const __amdgpu_buffer_rsrc_t r = scalar_rsrc(ptr, n * (int)row_bytes);
            const uint32_t at = __builtin_amdgcn_readfirstlane(to + place);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (SC_LDS void *)(uintptr_t)(at + i * 1024), 16, off[i], 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) put(row(i) < n && off[i] != OUT_OF_RANGE ? ptr + off[i] : nullptr, i);
        }
        ptr += 32 * row_bytes;
        advance();
    }
    // The next 32 rows of grouped query heads (row r is token token0 + r / group, head head0 +
    // r % group): row0 is the first.
    __device__ __forceinline__ void next_grouped(const Heads &a, const Heads &b, int64_t token0, int head0, uint32_t row0, uint32_t group)
    {
        const Heads &h = second ? b : a;
        const uint32_t t0 = row0 / group;
        const char *base = (const char *)h.p + ((token0 + t0) * h.row + head0 * h.head) * (int64_t)sizeof(T);
        const __amdgpu_buffer_rsrc_t rs = scalar_rsrc(base, 0x7fffffff);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t r = row0 + row(i), t = r / group;
            const bool there = row(i) < left && off[i] != OUT_OF_RANGE;
            if constexpr (DIRECT) {  // (the group's heads lie within 2^30 bytes)
                const uint32_t o = there ? (t - t0) * (uint32_t)(h.row * sizeof(T)) + (r - t * group) * (uint32_t)(h.head * sizeof(T)) + off[i]
                                         : OUT_OF_RANGE;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (SC_LDS void *)(uintptr_t)(to + place + i * 1024), 16, o, 0, 0, 0);
            } else {
                put(there ? base + ((int64_t)(t - t0) * h.row + (int64_t)(r - t * group) * h.head) * (int64_t)sizeof(T) + off[i] : nullptr, i);
            }
        }
        advance();
    }

  private:
    __device__ __forceinline__ int row(int i) const
    {
        return (int)(((__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % (WAVES / 2)) * PER * 1024 + i * 1024 + lane_id() * 16) / RB);
    }
    __device__ __forceinline__ void advance()
    {
        left -= 32;
        place = place == (RING - 1) * TILE ? 0 : place + TILE;
    }
    __device__ __forceinline__ void put(const char *from, int i) const
    {
        Raw16 v = {0, 0, 0, 0};
        if (from) v = *(const Raw16Any *)from;
        lds_write16(to + place + i * 1024 + lane_id() * 16, v);
    }
};

// --------------------------------------------------------------------------
// products
// --------------------------------------------------------------------------

// c += a b over one pair of pieces (8 bf16 or 4 fp32 of each half).
template <typename T>
__device__ __forceinline__ f32x16 mma_pieces(Raw16 a, Raw16 b, f32x16 c)
{
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
        return c;
    }
}

// Addresses of a lane's operand over the head dimension: row l % 32, piece 2j + a.
template <int RB>
struct HeadAddr {
    uint32_t at[RB / 32];
    __device__ __forceinline__ explicit HeadAddr(uint32_t lds)
    {
        const uint32_t l = lane_id();
#pragma unroll
        for (int j = 0; j < RB / 32; ++j) at[j] = lds + piece_at<RB>(l & 31, 2 * j + (l >> 5));
    }
    __device__ __forceinline__ void move(uint32_t by)
    {
#pragma unroll
        for (int j = 0; j < RB / 32; ++j) at[j] += by;
    }
};

// Addresses of a lane's transposed operand: row l % 32 of it is element 32 db + l % 32
// of the head; its columns are tile rows in the order of a result block's registers.
//   bf16: two 8-byte transposing reads give rows 4a .. 4a + 3 and 8 + 4a .. of 16.
//   fp32: one element of row 8 (i / 4) + 4 a + i % 4 at a time.
template <typename T, int RB>
struct RowsAddr;
template <int RB>
struct RowsAddr<uint16_t, RB> {
    static constexpr int DB = RB / 64;
    uint32_t at[2][DB];
    __device__ __forceinline__ explicit RowsAddr(uint32_t lds)
    {
        const uint32_t l = lane_id(), a = l >> 5, g = (l >> 4) & 1, t = l & 15;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int db = 0; db < DB; ++db)
                at[h][db] = lds + piece_at<RB>(8 * h + 4 * a + t / 4, db * 4 + g * 2 + (t & 3) / 2) + (t & 1) * 8;
    }
    __device__ __forceinline__ void move(uint32_t by)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int db = 0; db < DB; ++db) at[h][db] += by;
    }
};
template <int RB>
struct RowsAddr<float, RB> {
    static constexpr int DB = RB / 128;
    uint32_t at[8][DB];  // by i % 4 and bit 3 of the row; rows 16 apart share a swizzle
    __device__ __forceinline__ explicit RowsAddr(uint32_t lds)
    {
        const uint32_t l = lane_id(), a = l >> 5, d = l & 31;
#pragma unroll
        for (int h = 0; h < 8; ++h)
#pragma unroll
            for (int db = 0; db < DB; ++db)
                at[h][db] = lds + piece_at<RB>(8 * (h >> 2) + 4 * a + (h & 3), db * 8 + d / 4) + (d & 3) * 4;
    }
    __device__ __forceinline__ void move(uint32_t by)
    {
#pragma unroll
        for (int h = 0; h < 8; ++h)
#pragma unroll
            for (int db = 0; db < DB; ++db) at[h][db] += by;
    }
};

__device__ __forceinline__ u32x2 lds_read_tr(uint32_t at)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SC_LDS s16x4 *)(uintptr_t)at));
}

// Result registers 8h .. 8h + 7, rounded to bf16 (nearest even): the operand over 16 rows.
__device__ __forceinline__ Raw16 pack8(const f32x16 &s, int h)
{
    return Raw16{pack_bf16(s[8 * h], s[8 * h + 1]), pack_bf16(s[8 * h + 2], s[8 * h + 3]),
                 pack_bf16(s[8 * h + 4], s[8 * h + 5]), pack_bf16(s[8 * h + 6], s[8 * h + 7])};
}

// The result registers of a block of 32 rows as an operand over those rows.
template <typename T>
struct RowsOperand;
template <>
struct RowsOperand<uint16_t> {
    Raw16 v[2];
    __device__ __forceinline__ void set(const f32x16 &s)
    {
        v[0] = pack8(s, 0);
        v[1] = pack8(s, 1);
    }
};
template <>
struct RowsOperand<float> {
    f32x16 v;
    __device__ __forceinline__ void set(const f32x16 &s) { v = s; }
};

// The transposed operand of rows 16 (x / DB) .. + 15 and elements 32 (x % DB) .. + 31.
template <int RB>
__device__ __forceinline__ Raw16 rows_piece(const RowsAddr<uint16_t, RB> &ad, uint32_t at, int x)
{
    const int h = x / (RB / 64), db = x % (RB / 64);
    const u32x2 lo = lds_read_tr(ad.at[0][db] + at + 16 * h * RB), hi = lds_read_tr(ad.at[1][db] + at + 16 * h * RB);
    return Raw16{lo[0], lo[1], hi[0], hi[1]};
}

// The transposed operand of the rows of result register x / DB and elements 32 (x % DB) .. + 31.
template <int RB>
__device__ __forceinline__ float rows_piece(const RowsAddr<float, RB> &ad, uint32_t at, int x)
{
    const int i = x / (RB / 128), db = x % (RB / 128);
    return *(const SC_LDS float *)(uintptr_t)(ad.at[i & 7][db] + at + 16 * (i >> 3) * RB);
}

// acc[db] += transpose(32 tile rows) p, for every 32 elements db of the head; `at` is added to the
// addresses.
template <int RB>
__device__ __forceinline__ void mma_rows(const RowsAddr<uint16_t, RB> &ad, uint32_t at, const RowsOperand<uint16_t> &p,
                                         f32x16 (&acc)[RB / 64])
{
#pragma unroll
    for (int x = 0; x < 2 * (RB / 64); ++x)
        acc[x % (RB / 64)] = mma_pieces<uint16_t>(rows_piece<RB>(ad, at, x), p.v[x / (RB / 64)], acc[x % (RB / 64)]);
}
template <int RB>
__device__ __forceinline__ void mma_rows(const RowsAddr<float, RB> &ad, uint32_t at, const RowsOperand<float> &p,
                                         f32x16 (&acc)[RB / 128])
{
#pragma unroll
    for (int x = 0; x < 16 * (RB / 128); ++x)
        acc[x % (RB / 128)] = __builtin_amdgcn_mfma_f32_32x32x2f32(rows_piece<RB>(ad, at, x), p.v[x / (RB / 128)], acc[x % (RB / 128)], 0, 0, 0);
}

// The other half's value (lanes l and l ^ 32).
__device__ __forceinline__ float other_half(float v)
{
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(lane_id() < 32 ? r[1] : r[0]);
}

// Store row l % 32 of the transposed accumulators (elements of the head in registers),
// each value times `f`: the halves trade registers so that a lane holds 8 elements in a
// row, and write 16 bytes (bf16) or 32 bytes (fp32) at a time.
template <typename T, int DB>
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[DB], float f, T *row, int dim, bool valid)
{
    const int a = lane_id() >> 5;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // registers 8h .. 8h + 3 and 8h + 4 .. 8h + 7
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[db][8 * h + i] * f),
                                                          __float_as_uint(acc[db][8 * h + 4 + i] * f), false, false);
                v[i] = __uint_as_float(r[0]);
                v[4 + i] = __uint_as_float(r[1]);
            }
            const int e = 32 * db + 16 * h + 8 * a;
            if (!valid || e >= dim) continue;
            if constexpr (sizeof(T) == 2) {
                *(Raw16Any *)(row + e) = Raw16{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *(Raw16Any *)(row + e + 4 * i) = Raw16{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                                           __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
            }
        }
}

// Four elements of a row, each rounded once.
__device__ __forceinline__ void store4(float *p, f32x4 v) { *(Raw16Any *)p = __builtin_bit_cast(Raw16, v); }
__device__ __forceinline__ void store4(uint16_t *p, f32x4 v)
{
    const uint32_t a = pack_bf16(v[0], v[1]), b = pack_bf16(v[2], v[3]);
    p[0] = (uint16_t)a;
    p[1] = (uint16_t)(a >> 16);
    p[2] = (uint16_t)b;
    p[3] = (uint16_t)(b >> 16);
}

// Store into the output, of type T or fp32: `at` is the row's first element.
template <typename T, int DB>
__device__ __forceinline__ void store_out(const f32x16 (&acc)[DB], float f, void *out, bool f32, int64_t at, int dim, bool valid)
{
    if (sizeof(T) == 4 || f32) store_rows<float>(acc, f, (float *)out + at, dim, valid);
    else store_rows<T>(acc, f, (T *)out + at, dim, valid);
}
template <typename T>
__device__ __forceinline__ void store4_out(f32x4 v, void *out, bool f32, int64_t at)
{
    if (sizeof(T) == 4 || f32) store4((float *)out + at, v);
    else store4((T *)out + at, v);
}

// --------------------------------------------------------------------------
// arguments
// --------------------------------------------------------------------------

struct AttnArgs {
    Heads q, k, v, out, grad, dq, dk, dv;
    const int32_t *q_off, *k_off;
    int entries;
    int64_t nq, nk;
    int heads, kv_heads, group, dim;
    float scale;
    bool out_f32;  // out is fp32 beside bf16 tensors
    float *lse;    // [nq, heads]
    float *stat;   // [nq, heads, 2]: (base, delta) of a query row (backward)
    float *part;   // partial results of a split pass
    float *part2;
    int chunk;     // rows of the long side in one split
    int tiles;     // tiles of the short side taken by different blocks
    uint32_t slots;  // blocks that run at once, for cutting tiles (0: none are cut)
};

// Rows [beg, end) of `len` that a piece takes, in whole steps of 32.
__device__ __forceinline__ void piece_rows(const Work &w, int64_t len, int64_t *beg, int64_t *end)
{
    const int64_t steps = (len + 31) / 32;
    *beg = steps * w.piece / w.pieces * 32;
    *end = w.piece + 1 == w.pieces ? len : steps * (w.piece + 1) / w.pieces * 32;
}

// Compute units, and the blocks of 256 threads a unit holds at a time for tiles of `rb` bytes a
// row when registers allow `waves` a SIMD (LDS: two rings of four tiles of 32 rows).
constexpr int UNITS = 256;
constexpr int blocks_at_once(int rb, int waves) { return UNITS * (waves < 163840 / (256 * rb + 4096) ? waves : 163840 / (256 * rb + 4096)); }

// Whether tiles may be cut: a tile is long enough that a part of a round is worth the partial
// results and their join (some 20 us): on average 64 steps of the other side in bf16, 16
// in fp32, whose matrix products take eight times as long.
static inline bool cut_pays(int64_t other_rows, int entries, int dtype)
{
    return entries + 2 <= 64 * EACH && other_rows / entries >= (dtype == SUBMCONV_F32 ? 512 : 2048);
}

// How a pass is split along its long side: runs of `chunk` rows (0: not cut), at most
// `splits` of them in an entry, `tiles` tiles of the own side taken by different blocks.
struct SplitPlan {
    int chunk;
    int64_t splits;
    int tiles;
};
SplitPlan split_plan(int64_t own_rows, int own_tile, int64_t other_rows, int other_tile, int entries, int kv_heads, int64_t slots,
                     int dtype);

}  // namespace sc
