// Softmax attention over ragged batches, forward.
//
//   s_j = scale q . k_j over the keys j of the query's entry,  p = softmax(s),  o = sum_j p_j v_j
//
// One pass over the keys with a running maximum m and sum l: a tile's weights are
// exp(s - m); when a tile's maximum passes m, what was summed so far is scaled by
// exp(m_old - m_new).  A query without keys gives zeros (and lse = -inf).
//
// A wave owns 32 query rows (token, head of the key head's group): queries stay in
// registers as the second operand of s^T = k q^T, the result registers become the
// second operand of o^T += v^T p^T.  A block's four waves share tiles of keys and
// values in LDS.
//
// 12,948 x 12 x 128 bf16: 1.04 ms, 990 TFLOP/s (a library product of 8192^3 reaches 1124 to
// 1136); 32,768 x 12 x 128: 1051.  Bound by what two waves of a SIMD issue: the
// matrix pipe is busy about half the time, the softmax's arithmetic takes most of the
// rest, and one does not hide all of the other.  64 query rows a wave (half the LDS reads)
// need more registers than there are for two waves and ran 2.7 times as long; eight
// waves to a block (half the copies) changed nothing.
#include "attention.h"

namespace sc {

// What a row's running maximum may be passed by, in powers of two, before the sums are
// rescaled: weights stay below 2^8, far from overflow, and most tiles skip the rescaling.
constexpr float SLACK = 8.0f;

// A weight is exp2(s c - base) with c = scale log2(e), m the row's running maximum and base = m c
// rounded to fp32: one fused rounding of the difference.  What the rounding of m c leaves
// is a common factor of the row's weights and their sum, so everything that follows has to
// use that same rounded number: the product is kept out of any fused operation (contraction
// would make base - next_base a fused m c - next_base, off by up to 2^5 in the exponent).
// Past this size of m c that common factor could overflow (and m c itself); the weight is
// then exp2((s - m) c), where equal scores cancel exactly.
constexpr float HUGE_BASE = 1073741824.0f;
__device__ __forceinline__ float rounded_product(float m, float c)
{
#pragma clang fp contract(off)
    return m * c;
}
__device__ __forceinline__ bool huge(float m, float c) { return m != -INFINITY && !(fabsf(m * c) <= HUGE_BASE); }
__device__ __forceinline__ float base_of(float m, float c) { return m == -INFINITY || huge(m, c) ? 0.0f : rounded_product(m, c); }

// What sums relative to the maximum m are worth relative to next >= m: exactly 1 where the
// maximum is the same.  Where just one of the two is huge, its m c is meant exactly.
__device__ __forceinline__ float rescale(float m, float next, float c)
{
    if (m == next) return 1.0f;
    if (m == -INFINITY) return 0.0f;  // nothing is summed yet
    float e = base_of(m, c) - base_of(next, c);
    if (huge(m, c)) e = huge(next, c) ? (m - next) * c : fmaf(m, c, -base_of(next, c));
    else if (huge(next, c)) e = -fmaf(next, c, -base_of(m, c));
    return __builtin_amdgcn_exp2f(e);
}

// log sum exp from the maximum and the sum of the weights.
__device__ __forceinline__ float log_sum(float m, float l, float scale)
{
    if (l == 0.0f) return -INFINITY;  // no key, or none with a finite score
    const float c = scale * LOG2E, e = __builtin_amdgcn_logf(l);
    return huge(m, c) ? m * scale + e * LN2 : (base_of(m, c) + e) * LN2;
}

// acc *= f where `on`, in place.  One straight piece of code for the compiler: a branch
// around the products makes it keep every accumulator twice and copy them where the
// branch is not taken, which is nearly always.  The waits cover a matrix product that is
// still writing acc, and one that reads it next.
__device__ __forceinline__ void scale_if(f32x16 &acc, float f, uint64_t on)
{
    asm volatile("s_cmp_eq_u64 %17, 0\n\t"
                 "s_cbranch_scc1 .Lkeep%=\n\t"
                 "s_nop 15\n\ts_nop 15\n\t"
                 "v_mul_f32 %0, %16, %0\n\tv_mul_f32 %1, %16, %1\n\tv_mul_f32 %2, %16, %2\n\tv_mul_f32 %3, %16, %3\n\t"
                 "v_mul_f32 %4, %16, %4\n\tv_mul_f32 %5, %16, %5\n\tv_mul_f32 %6, %16, %6\n\tv_mul_f32 %7, %16, %7\n\t"
                 "v_mul_f32 %8, %16, %8\n\tv_mul_f32 %9, %16, %9\n\tv_mul_f32 %10, %16, %10\n\tv_mul_f32 %11, %16, %11\n\t"
                 "v_mul_f32 %12, %16, %12\n\tv_mul_f32 %13, %16, %13\n\tv_mul_f32 %14, %16, %14\n\tv_mul_f32 %15, %16, %15\n\t"
                 "s_nop 7\n"
                 ".Lkeep%=:"
                 : "+v"(acc[0]), "+v"(acc[1]), "+v"(acc[2]), "+v"(acc[3]), "+v"(acc[4]), "+v"(acc[5]), "+v"(acc[6]),
                   "+v"(acc[7]), "+v"(acc[8]), "+v"(acc[9]), "+v"(acc[10]), "+v"(acc[11]), "+v"(acc[12]), "+v"(acc[13]),
                   "+v"(acc[14]), "+v"(acc[15])
                 : "v"(f), "s"(on)
                 : "scc");
}

constexpr int FWD_WAVES = 4, RING = 4;

// A step handles 32 keys.  Its wave has the scores of its own keys in registers already,
// and, while it turns them into weights, the matrix cores form the scores of the next
// 32 keys; then they take the weights' product with the values, and the next scores'
// maximum is found meanwhile.  Keys and values are copied three steps ahead, into rings of
// four tiles in LDS.
//
// SPLIT: a block takes one run of `chunk` keys of
// an entry and leaves (sum, m, l) of it in part / part2 for k_attn_join; otherwise a block
// takes one tile of query rows over all keys.
constexpr int fwd_residency(int rb) { return rb > 256 ? 1 : rb > 128 ? 2 : rb > 64 ? 3 : 4; }  // waves a SIMD

template <typename T, int DP, bool SPLIT, bool DIRECT>
__global__ __launch_bounds__(64 * FWD_WAVES, fwd_residency(DP * sizeof(T))) void k_attn(AttnArgs A)
{
    constexpr int RB = DP * (int)sizeof(T), NJ = RB / 32, DB = DP / 32, TILE = 32 * RB, ROWS = 32 * FWD_WAVES;
    constexpr uint32_t V0 = RING * TILE;  // the values' ring
    __shared__ __attribute__((aligned(1024))) char smem[2 * RING * TILE];
    const uint32_t lds = (uint32_t)(uintptr_t)(SC_LDS char *)smem;

    const Ragged rq = {A.q_off, A.entries, A.nq, A.group}, rk = {A.k_off, A.entries, A.nk, 1};
    Work w;
    int64_t qtile, key0 = 0, split = 0;
    if constexpr (SPLIT) {
        if (!find_work(rk, rq, A.chunk, xcd_work(), A.kv_heads * A.tiles, 0, false, &w) || !w.real) return;
        split = w.tile;
        key0 = split * A.chunk;
        qtile = w.which % A.tiles;
        w.which /= A.tiles;
    } else {
        if (!find_work(rq, rk, ROWS, xcd_work(), A.kv_heads, A.slots, false, &w)) return;
        qtile = w.tile;
    }
    const int hk = (int)w.which;
    const int64_t q_beg = SPLIT ? w.other_beg : w.own_beg, k_beg = SPLIT ? w.own_beg : w.other_beg;
    const int64_t rows = (SPLIT ? w.other_len : w.own_len) * A.group;
    int64_t keys64 = (SPLIT ? w.own_len : w.other_len) - key0;
    if (SPLIT && keys64 <= 0) return;  // a number without a run (see first_tile)
    if (SPLIT && keys64 > A.chunk) keys64 = A.chunk;
    if (!SPLIT && w.pieces > 1) {
        piece_rows(w, w.other_len, &key0, &keys64);
        keys64 -= key0;
    }
    const int keys = (int)keys64, steps = (keys + 31) / 32;

    const int lane = lane_id(), half = lane >> 5;
    const float c = A.scale * LOG2E;
    const T *kp = (const T *)A.k.p + (k_beg + key0) * A.k.row + hk * A.k.head;
    const T *vp = (const T *)A.v.p + (k_beg + key0) * A.v.row + hk * A.v.head;
    Fill<T, RB, FWD_WAVES, RING, DIRECT> fill;
    fill.init(lds, lds + V0, A.k.row, A.v.row, A.dim);
    HeadAddr<RB> ka(lds);
    RowsAddr<T, RB> va(lds + V0);

    for (; qtile * ROWS < rows; qtile += SPLIT ? A.tiles : rows) {
        const int64_t wave_row = qtile * ROWS + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 32;
        if (SPLIT) __syncthreads();  // the rings' last readers are done
        fill.start(kp, vp, keys);
        // keys 0 .. 2 and values 0 .. 1; then, before every pair of steps u, u + 1, keys u + 3 and
        // u + 4 and values u + 2 and u + 3, whose places were last read in the pair before
        if (steps)
            for (int u = fill.second; u < 3; ++u) fill.next();
        if (wave_row >= rows) {  // a wave past the entry's rows only helps with the copies
            if (steps) {
                wait_copies_and_barrier<0>();
                wait_copies_and_barrier<0>();
                for (int u = 0; u + 2 < steps; u += 2) {
                    fill.next();
                    fill.next();
                    wait_copies_and_barrier<0>();
                }
            }
            continue;
        }

        Raw16 q[NJ];
        const uint32_t row = (uint32_t)(wave_row + (lane & 31)), token = A.group == 1 ? row : row / A.group;
        const int head = hk * A.group + (int)(row - token * A.group);
        const bool valid = row < rows;
        const T *qp = (const T *)A.q.p + (q_beg + token) * A.q.row + head * A.q.head;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = (2 * j + half) * VEC<T>;
            q[j] = Raw16{0, 0, 0, 0};
            if (valid && e < A.dim) q[j] = *(const Raw16Any *)(qp + e);
        }
        f32x16 o[DB], s[2];
        float m = -INFINITY, l = 0.0f, base = 0.0f;
        uint64_t big = 0;  // some row's maximum is huge
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] = f32x16{};

        // scores of the keys in ring place `at`
        auto scores = [&](f32x16 &t, uint32_t at) {
            t = f32x16{};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const Raw16 k = lds_read16(ka.at[j] + at);
                t = mma_pieces<T>(k, q[j], t);
            }
        };
        // scores of step u past the last key are none
        auto mask = [&](f32x16 &t, int u) {
            if (__builtin_expect(keys - u * 32 < 32, 0)) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (8 * (i / 4) + 4 * half + i % 4 >= keys - u * 32) t[i] = -INFINITY;
            }
        };
        // with the scores' maximum of this half's keys, everything their weights need
        auto settle = [&](f32x16 &t, float &top) {
            float f = 1.0f;
            top = fmaxf(top, other_half(top));
            const uint64_t any = __ballot((top - m) * c > SLACK);
            if (__builtin_expect(any != 0, 0)) {
                const float next = fmaxf(m, top);
                f = rescale(m, next, c);
                m = next;
                l *= f;
                base = base_of(next, c);  // (0 for -inf: weights are exp(-inf))
                big = __ballot(huge(next, c));
            }
#pragma unroll
            for (int db = 0; db < DB; ++db) scale_if(o[db], f, any);
            if (__builtin_expect(big != 0, 0)) {  // differences of scores in the scores' place
                const bool mine = huge(m, c);
#pragma unroll
                for (int i = 0; i < 16; ++i) t[i] = mine ? t[i] - m : t[i];
            }
        };
        auto maximum = [&](const f32x16 &t, float &top, int from, int to) {
#pragma unroll
            for (int i = from; i < to; ++i) top = i ? fmaxf(top, t[i]) : t[i];
        };
        auto weights = [&](f32x16 &t, int from, int to) {
#pragma unroll
            for (int i = from; i < to; ++i) {
                t[i] = __builtin_amdgcn_exp2f(fmaf(t[i], c, -base));
                l += t[i];
            }
        };
        auto product = [&](f32x16 &t, uint32_t vat) {
            RowsOperand<T> p;
            p.set(t);
            mma_rows<RB>(va, vat, p, o);
        };
        // step u from scores t, leaving the next step's in n; kat, vat: the tiles' places past ka and va
        auto step = [&](f32x16 &t, f32x16 &n, int u, uint32_t kat, uint32_t vat) {
            float top;
            if constexpr (sizeof(T) == 2) {
                // in the order it is to run: LDS reads AHEAD of their use, and between the matrix
                // products a piece of the arithmetic; first the scores with half the weights, then
                // their product with the values, with the other half and the maximum
                constexpr int AHEAD = NJ < 4 ? NJ : 4;
                Raw16 k[NJ], v[2 * DB], p[2];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) k[j] = lds_read16(ka.at[j] + kat);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (j + AHEAD < NJ) k[j + AHEAD] = lds_read16(ka.at[j + AHEAD] + kat);
                    else if (j + AHEAD - NJ < 2 && j + AHEAD - NJ < 2 * DB) v[j + AHEAD - NJ] = rows_piece<RB>(va, vat, j + AHEAD - NJ);
                    n = mma_pieces<T>(k[j], q[j], j ? n : f32x16{});
                    weights(t, 8 * j / NJ, 8 * (j + 1) / NJ);
                    __builtin_amdgcn_sched_barrier(0);
                }
                p[0] = pack8(t, 0);
                mask(n, u + 1);
#pragma unroll
                for (int x = 0; x < 2 * DB; ++x) {
                    const int h = x / DB, db = x % DB;
                    if (x + 2 < 2 * DB) v[x + 2] = rows_piece<RB>(va, vat, x + 2);
                    o[db] = mma_pieces<T>(v[x], p[h], o[db]);
                    if (h == 0) weights(t, 8 + 8 * db / DB, 8 + 8 * (db + 1) / DB);
                    else maximum(n, top, 16 * db / DB, 16 * (db + 1) / DB);
                    if (x == DB - 1) p[1] = pack8(t, 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                // the same; a weight is an operand as it is, so the second half is made as the product goes
                constexpr int AHEAD = NJ < 2 ? NJ : 2, FAR = 8;
                Raw16 k[NJ];
                float v[16 * DB];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) k[j] = lds_read16(ka.at[j] + kat);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (j + AHEAD < NJ) k[j + AHEAD] = lds_read16(ka.at[j + AHEAD] + kat);
                    else {
#pragma unroll
                        for (int x = 0; x < FAR / AHEAD; ++x)
                            v[(j + AHEAD - NJ) * (FAR / AHEAD) + x] = rows_piece<RB>(va, vat, (j + AHEAD - NJ) * (FAR / AHEAD) + x);
                    }
                    n = mma_pieces<T>(k[j], q[j], j ? n : f32x16{});
                    weights(t, 8 * j / NJ, 8 * (j + 1) / NJ);
                    __builtin_amdgcn_sched_barrier(0);
                }
                mask(n, u + 1);
#pragma unroll
                for (int x = 0; x < 16 * DB; ++x) {
                    const int i = x / DB, db = x % DB;
                    if (x + FAR < 16 * DB) v[x + FAR] = rows_piece<RB>(va, vat, x + FAR);
                    o[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(v[x], t[i], o[db], 0, 0, 0);
                    if (db == 0) {
                        if (i < 8) weights(t, 8 + i, 9 + i);
                        else maximum(n, top, 2 * (i - 8), 2 * (i - 8) + 2);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            settle(n, top);
        };

        if (steps) {
            wait_copies_and_barrier<0>();
            float top;
            scores(s[0], 0);
            mask(s[0], 0);
            maximum(s[0], top, 0, 16);
            settle(s[0], top);
            wait_copies_and_barrier<0>();
            int u = 0;
            for (; u + 2 < steps; u += 2) {  // ring places u mod 4 = 0 or 2: the addresses move to the other half
                const uint32_t other = u & 2 ? -2 * TILE : 2 * TILE;
                fill.next();
                fill.next();
                step(s[0], s[1], u, TILE, 0);
                ka.move(other);
                step(s[1], s[0], u + 1, 0, TILE);
                va.move(other);
                wait_copies_and_barrier<0>();
            }
            if (u + 1 < steps) {
                step(s[0], s[1], u, TILE, 0);
                weights(s[1], 0, 16);
                product(s[1], TILE);
            } else {
                weights(s[0], 0, 16);
                product(s[0], 0);
            }
            if (u & 2) {
                ka.move(-2 * TILE);
                va.move(-2 * TILE);
            }
        }
        const float sum = l + other_half(l);
        if constexpr (SPLIT) {
            const int64_t at = split * A.nq * A.heads + (q_beg + token) * A.heads + head;
            store_rows<float>(o, 1.0f, A.part + at * A.dim, A.dim, valid);
            if (valid && half == 0) *(float2 *)(A.part2 + 2 * at) = make_float2(m, sum);
        } else if (w.pieces > 1) {
            const int64_t at = (int64_t)w.index * ROWS + (threadIdx.x >> 6) * 32 + (lane & 31);
            store_rows<float>(o, 1.0f, A.part + at * A.dim, A.dim, valid);
            if (valid && half == 0) *(float2 *)(A.part2 + 2 * at) = make_float2(m, sum);
        } else {
            store_out<T>(o, sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum), (void *)A.out.p, A.out_f32,
                         (q_beg + token) * A.out.row + head * A.out.head, A.dim, valid);
            if (A.lse && valid && half == 0) A.lse[(q_beg + token) * A.heads + head] = log_sum(m, sum, A.scale);
        }
    }
}

// Every variant that is launched, spelled out: the host pass leaves some of them out when they
// are only named in a launch.
#define VARIANTS(T, DP, DIRECT) \
    template __global__ void k_attn<T, DP, false, DIRECT>(AttnArgs); \
    template __global__ void k_attn<T, DP, true, DIRECT>(AttnArgs);
VARIANTS(float, 32, true)
VARIANTS(float, 64, true)
VARIANTS(float, 96, true)
VARIANTS(float, 128, true)
VARIANTS(float, 128, false)
VARIANTS(uint16_t, 32, true)
VARIANTS(uint16_t, 64, true)
VARIANTS(uint16_t, 96, true)
VARIANTS(uint16_t, 128, true)
VARIANTS(uint16_t, 128, false)
#undef VARIANTS

// The splits' sums of a query row joined, in a fixed order, by A.tiles of a block's four
// waves (four rows a block, or one where there are many splits).
constexpr int JOIN_MAX_SPLITS = 2048, JOIN_WAVES = 4, JOIN_WAVE_SPLITS = 64;
template <typename T>
__global__ __launch_bounds__(64 * JOIN_WAVES) void k_attn_join(AttnArgs A)
{
    __shared__ f32x4 acc[JOIN_WAVES][64];
    __shared__ float part_l[JOIN_WAVES], weights[JOIN_MAX_SPLITS];
    const int lane = lane_id(), wave = threadIdx.x >> 6, mine = wave % A.tiles, first = wave - mine;
    const int64_t rows = A.nq * A.heads, at = (int64_t)blockIdx.x * (JOIN_WAVES / A.tiles) + wave / A.tiles;
    const bool on = at < rows;
    const int64_t token = on ? at / A.heads : 0;
    const int head = (int)(at - token * A.heads);
    const Ragged rq = {A.q_off, A.entries, A.nq, 1}, rk = {A.k_off, A.entries, A.nk, 1};
    const int part = find_part(rq, token);
    const bool real = part >= 1 && part <= A.entries;
    const int64_t keys = real && on ? rk.bound(part + 1) - rk.bound(part) : 0;
    const int n = keys > 0 ? (int)((keys + A.chunk - 1) / A.chunk) : 0;
    const float c = A.scale * LOG2E;

    float top = -INFINITY;
    for (int s = lane; s < n; s += 64) top = fmaxf(top, A.part2[2 * (s * rows + at)]);
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    float l = 0.0f, *weight = weights + (A.tiles == 1 ? wave * JOIN_WAVE_SPLITS : 0);
    for (int s = lane + 64 * mine; s < n; s += 64 * A.tiles) {
        const float2 ml = *(const float2 *)(A.part2 + 2 * (s * rows + at));
        weight[s] = rescale(ml.x, top, c);
        l += ml.y * weight[s];
    }
    __syncthreads();
    const int pieces = A.dim / 4, groups = 64 / pieces, g = lane / pieces, e = lane % pieces;
    f32x4 sum = {0, 0, 0, 0};
    if (g < groups) {
#pragma unroll 8
        for (int s = g + groups * mine; s < n; s += groups * A.tiles)
            sum += *(const f32x4 *)(A.part + (s * rows + at) * A.dim + 4 * e) * weight[s];
    }
    l = lanes_sum<64>(l);
    acc[wave][lane] = sum;
    if (lane == 0) part_l[wave] = l;
    __syncthreads();
    if (!on || mine || g) return;
    for (int i = 1; i < groups * A.tiles; ++i) sum += acc[first + i / groups][i % groups * pieces + e];
    for (int i = 1; i < A.tiles; ++i) l += part_l[first + i];
    sum *= l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    store4_out<T>(sum, (void *)A.out.p, A.out_f32, token * A.out.row + head * A.out.head + 4 * e);
    if (A.lse && e == 0) A.lse[at] = log_sum(top, l, A.scale);
}

// The pieces of cut tiles joined: blockIdx.x counts the tiles, blockIdx.y their quarters.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_join_cut(AttnArgs A)
{
    constexpr int ROWS = 32 * FWD_WAVES;
    const Ragged rq = {A.q_off, A.entries, A.nq, A.group}, rk = {A.k_off, A.entries, A.nk, 1};
    Work w;
    if (!find_work(rq, rk, ROWS, blockIdx.x, A.kv_heads, A.slots, true, &w)) return;
    const int pieces = A.dim / 4, groups = 256 / pieces, g = threadIdx.x / pieces, e = threadIdx.x % pieces;
    const int64_t rows = w.own_len * A.group - w.tile * ROWS;  // of this tile on
    if (g >= groups) return;
    for (int r = blockIdx.y * (ROWS / 4) + g; r < (int)(blockIdx.y + 1) * (ROWS / 4) && r < rows; r += groups) {
        const uint32_t row = (uint32_t)(w.tile * ROWS) + r, token = A.group == 1 ? row : row / A.group;
        const int head = (int)(w.which * A.group + (row - token * A.group));
        const int64_t first = (int64_t)w.index * ROWS + r;
        float2 ml[MAX_PIECES];
        f32x4 v[MAX_PIECES];
        float top = -INFINITY, l = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < MAX_PIECES; ++i) {
            ml[i] = make_float2(-INFINITY, 0.0f);
            v[i] = f32x4{0, 0, 0, 0};
            if (i < w.pieces) {
                ml[i] = *(const float2 *)(A.part2 + 2 * (first + i * ROWS));
                v[i] = *(const f32x4 *)(A.part + (first + i * ROWS) * A.dim + 4 * e);
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < MAX_PIECES; ++i) top = fmaxf(top, ml[i].x);
        f32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (uint32_t i = 0; i < MAX_PIECES; ++i)
            if (i < w.pieces) {
                const float f = rescale(ml[i].x, top, A.scale * LOG2E);
                l += ml[i].y * f;
                sum += v[i] * f;
            }
        sum *= l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        store4_out<T>(sum, (void *)A.out.p, A.out_f32, (w.own_beg + token) * A.out.row + head * A.out.head + 4 * e);
        if (A.lse && e == 0) A.lse[(w.own_beg + token) * A.heads + head] = log_sum(top, l, A.scale);
    }
}

// How a pass over a long side is split when its own side has few tiles, so few that they and
// half as many more would still run at once (`slots` blocks do): into runs of at least
// MIN_CHUNK rows, WANT_BLOCKS blocks in all, several to each place, since the entries and
// the last runs are not alike (measured on 20384 x 4111 rows, 4 heads of 64, fp32, for the keys'
// gradients: 768 blocks 538 us, 1536 466, 3072 490).  chunk = 0: not at all, as in bf16 where
// the other side is so short that the join's launch costs more than the split saves (64
// queries of 4 x 64: 512 keys 18.8 us split, 16.3 whole; 1024 keys 19.2 and 20.4).  The limit
// lies between those two; among several entries the longest sets the time, some times the
// average, so it is lower (7 entries, 611 keys on average, 1904 the longest: 20.4 and 31.3).
// fp32 has no such limit: 64 queries over 256 keys take 21.8 us split and 24.3 whole.
constexpr int64_t WANT_BLOCKS = 1536, MIN_CHUNK = 64;

SplitPlan split_plan(int64_t own_rows, int own_tile, int64_t other_rows, int other_tile, int entries, int kv_heads, int64_t slots,
                     int dtype)
{
    SplitPlan p = {0, 0, 1};
    if (own_rows == 0 || other_rows == 0) return p;
    if (dtype == SUBMCONV_BF16 && other_rows / entries < (entries == 1 ? 768 : 512)) return p;
    const int64_t per_entry = (own_rows / entries + own_tile - 1) / own_tile;
    int64_t tiles = per_entry > 0 ? per_entry : 1;
    const int64_t used = entries < own_rows ? entries : own_rows;
    if (tiles * used * kv_heads * 3 > slots * 2) return p;
    int64_t runs = WANT_BLOCKS / (tiles * kv_heads);
    if (runs > JOIN_MAX_SPLITS - 1) runs = JOIN_MAX_SPLITS - 1;
    int64_t chunk = (other_rows + runs - 1) / runs;
    if (chunk < MIN_CHUNK) chunk = MIN_CHUNK;
    chunk = (chunk + other_tile - 1) / other_tile * other_tile;
    if (chunk * 2 > other_rows / entries || chunk > (1 << 30)) return p;  // entries of one run or two: nothing to gain
    p.chunk = (int)chunk;
    p.splits = (other_rows + chunk - 1) / chunk;
    // an entry longer than the average has more tiles, and a block that takes two takes twice as long
    if (entries > 1 && tiles > 1) tiles *= 2;
    p.tiles = (int)tiles;
    return p;
}

// Blocks that run at once.
static int fwd_slots(const AttnArgs &A, int dtype)
{
    const int rb = (A.dim + 31) / 32 * 32 * (dtype == SUBMCONV_F32 ? 4 : 2);
    return blocks_at_once(rb, fwd_residency(rb));
}

static SplitPlan fwd_plan(const AttnArgs &A, int dtype)
{
    return split_plan(A.nq * A.group, 32 * FWD_WAVES, A.nk, 32, A.entries, A.kv_heads, fwd_slots(A, dtype), dtype);
}

// The same where tiles may be cut, else 0.
static uint32_t fwd_cut(const AttnArgs &A, int dtype) { return cut_pays(A.nk, A.entries, dtype) ? (uint32_t)fwd_slots(A, dtype) : 0; }

size_t attention_workspace(const AttnArgs &A, int dtype)
{
    const SplitPlan p = fwd_plan(A, dtype);
    const size_t rows = p.chunk ? (size_t)p.splits * A.nq * A.heads : (size_t)2 * fwd_cut(A, dtype) * 32 * FWD_WAVES;
    return rows * (A.dim + 2) * sizeof(float);
}

// Whether keys and values can be copied straight into LDS (see Fill).
static bool direct(const AttnArgs &A, int es)
{
    return !(((uintptr_t)A.k.p | (uintptr_t)A.v.p | (uintptr_t)((A.k.row | A.v.row | A.k.head | A.v.head) * es)) & 15) &&
           A.k.row >= A.dim && A.v.row >= A.dim;
}

template <typename T, int DP, bool DIRECT>
static int run_fwd(AttnArgs A, const SplitPlan &p, void *workspace, hipStream_t st)
{
    const dim3 block(64 * FWD_WAVES);
    if (p.chunk) {
        A.chunk = p.chunk;
        A.tiles = p.tiles;
        A.part = (float *)workspace;
        A.part2 = A.part + p.splits * A.nq * A.heads * A.dim;
        const int64_t work = ragged_tiles(A.nk, A.entries, 1, p.chunk) * A.kv_heads * p.tiles;
        hipLaunchKernelGGL((k_attn<T, DP, true, DIRECT>), dim3(xcd_grid(work)), block, 0, st, A);
        SC_LAUNCHED("attention (split)");
        A.tiles = p.splits > JOIN_WAVE_SPLITS ? JOIN_WAVES : 1;
        const int64_t per = JOIN_WAVES / A.tiles;
        hipLaunchKernelGGL((k_attn_join<T>), dim3((unsigned)((A.nq * A.heads + per - 1) / per)), dim3(64 * JOIN_WAVES), 0, st, A);
        SC_LAUNCHED("attention join");
        return SUBMCONV_OK;
    }
    A.slots = DIRECT ? fwd_cut(A, sizeof(T) == 4 ? SUBMCONV_F32 : SUBMCONV_BF16) : 0;
    A.part = (float *)workspace;
    A.part2 = A.part + (size_t)2 * A.slots * 32 * FWD_WAVES * A.dim;
    const int64_t work = ragged_tiles(A.nq, A.entries, A.group, 32 * FWD_WAVES) * A.kv_heads + 2 * A.slots;
    hipLaunchKernelGGL((k_attn<T, DP, false, DIRECT>), dim3(xcd_grid(work)), block, 0, st, A);
    SC_LAUNCHED("attention");
    if (A.slots) {
        hipLaunchKernelGGL(k_attn_join_cut<T>, dim3(A.slots, 4), dim3(256), 0, st, A);
        SC_LAUNCHED("attention join of cut tiles");
    }
    return SUBMCONV_OK;
}

int attention(const AttnArgs &A, int dtype, void *workspace, hipStream_t st)
{
    const SplitPlan p = fwd_plan(A, dtype);
    const int dp = (A.dim + 31) / 32;
#define GO(T)                                                                                       \
    if (!direct(A, sizeof(T))) return run_fwd<T, 128, false>(A, p, workspace, st); \
    switch (dp) {                                                                                   \
    case 1: return run_fwd<T, 32, true>(A, p, workspace, st); \
    case 2: return run_fwd<T, 64, true>(A, p, workspace, st); \
    case 3: return run_fwd<T, 96, true>(A, p, workspace, st); \
    default: return run_fwd<T, 128, true>(A, p, workspace, st); \
    }
    if (dtype == SUBMCONV_F32) {
        GO(float)
    } else {
        GO(uint16_t)
    }
#undef GO
}

}  // namespace sc
