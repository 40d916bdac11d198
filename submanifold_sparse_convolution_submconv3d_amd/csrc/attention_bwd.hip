// Softmax attention over ragged batches, backward.
//
// With p = exp(scale q k - lse), g the gradient of o and delta = sum_d g o (per query):
//
//   dp = g v,  ds = p (dp - delta),  dv = sum_q p g,  dk = scale sum_q ds q,  dq = scale sum_k ds k
//
// Two kernels, each forming p and ds again: k_attn_dq owns queries and walks the keys (3
// products), k_attn_dkv owns keys and walks the query rows of all heads that share them
// (4 products).  Seven products instead of the five of one kernel, but every gradient is
// summed in registers in a fixed order: no atomics, equal calls give equal bits, and a
// shared key head's gradient needs no second pass over its query heads.
#include "attention.h"

namespace sc {

constexpr int BWD_WAVES = 4, BWD_ROWS = 32 * BWD_WAVES, RING = 4;

// A score's exponent is s c - base; a query whose scores are all -inf has lse = -inf and
// weights exp(-inf), so its base must be finite.
__device__ __forceinline__ float lse_base(float lse) { return lse == -INFINITY ? 0.0f : lse * LOG2E; }

// A step handles 32 keys: the matrix cores form s^T = k q^T and dp^T = v g^T of the next
// keys while ds of its own is computed, then add k^T ds.  Keys and values are copied three
// steps ahead into rings of four tiles in LDS.  Leaves (base, delta) of every query
// row for k_attn_dkv.  delta comes from out as it is stored: forming it as sum_k p dp instead would
// take another product here (dq needs sum_k p k to be set right afterwards); a caller to whom
// the rounding of a bf16 out matters keeps it in fp32.  7042 + 5906 rows x 8 x 128 bf16: 468 us,
// 1.11 PFLOP/s of its three products, with 56 registers spilled (two waves a SIMD leave 256).
// 8000 x 4 x 128 fp32: 1.51 ms, 130 TFLOP/s (a library product of 8192^3 reaches 151).
constexpr int dq_residency(int rb) { return rb > 256 ? 1 : 2; }  // waves a SIMD

template <typename T, int DP, bool SPLIT, bool DIRECT>
__global__ __launch_bounds__(64 * BWD_WAVES, dq_residency(DP * sizeof(T))) void k_attn_dq(AttnArgs A)
{
    constexpr int RB = DP * (int)sizeof(T), NJ = RB / 32, DB = DP / 32, TILE = 32 * RB;
    constexpr uint32_t V0 = RING * TILE;
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
        if (!find_work(rq, rk, BWD_ROWS, xcd_work(), A.kv_heads, A.slots, false, &w)) return;
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
    Fill<T, RB, BWD_WAVES, RING, DIRECT> fill;
    constexpr int PER = Fill<T, RB, BWD_WAVES, RING, DIRECT>::PER;
    fill.init(lds, lds + V0, A.k.row, A.v.row, A.dim);
    HeadAddr<RB> ka(lds);
    RowsAddr<T, RB> kt(lds);

    for (; qtile * BWD_ROWS < rows; qtile += SPLIT ? A.tiles : rows) {
        const int64_t wave_row = qtile * BWD_ROWS + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 32;
        if (SPLIT) __syncthreads();
        fill.start(kp, vp, keys);
        if (steps)
            for (int u = 1; u < RING; ++u) fill.next();
        if (wave_row >= rows) {  // a wave past the entry's rows only helps with the copies
            if (steps) {
                wait_copies_and_barrier<2 * PER>();
                for (int u = 0; u < steps; ++u) {
                    if (u) fill.next();
                    wait_copies_and_barrier<PER>();
                }
                wait_copies_and_barrier<0>();
            }
            continue;
        }
        const uint32_t row = (uint32_t)(wave_row + (lane & 31)), token = A.group == 1 ? row : row / A.group;
        const int head = hk * A.group + (int)(row - token * A.group);
        const bool valid = row < rows;
        const int64_t at = (q_beg + token) * A.heads + head;
        Raw16 q[NJ], g[NJ];
        float base = 0.0f, delta = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) q[j] = g[j] = Raw16{0, 0, 0, 0};
        if (valid) {
            const T *qp = (const T *)A.q.p + (q_beg + token) * A.q.row + head * A.q.head;
            const T *gp = (const T *)A.grad.p + (q_beg + token) * A.grad.row + head * A.grad.head;
            const int64_t o = (q_beg + token) * A.out.row + head * A.out.head;
            base = lse_base(A.lse[at]);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int e = (2 * j + half) * VEC<T>;
                if (e >= A.dim) continue;
                q[j] = *(const Raw16Any *)(qp + e);
                g[j] = *(const Raw16Any *)(gp + e);
                float a[VEC<T>], b[VEC<T>];
                unpack(g[j], a, gp);
                if (sizeof(T) == 2 && A.out_f32) {
#pragma unroll
                    for (int i = 0; i < VEC<T>; ++i) b[i] = ((const float *)A.out.p)[o + e + i];
                } else {
                    unpack((Raw16) * (const Raw16Any *)((const T *)A.out.p + o + e), b, gp);
                }
#pragma unroll
                for (int i = 0; i < VEC<T>; ++i) delta += a[i] * b[i];
            }
        }
        delta += other_half(delta);
        if (valid && half == 0 && split == 0 && w.piece == 0) *(float2 *)(A.stat + 2 * at) = make_float2(base, delta);

        f32x16 dq[DB], s[2], dp[2];
#pragma unroll
        for (int db = 0; db < DB; ++db) dq[db] = f32x16{};
        auto products = [&](f32x16 &t, f32x16 &e, uint32_t place) {
            t = e = f32x16{};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                t = mma_pieces<T>(lds_read16(ka.at[j] + place), q[j], t);
                e = mma_pieces<T>(lds_read16(ka.at[j] + place + V0), g[j], e);
            }
        };
        auto mask = [&](f32x16 &t, int u) {
            if (__builtin_expect(keys - u * 32 < 32, 0)) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (8 * (i / 4) + 4 * half + i % 4 >= keys - u * 32) t[i] = -INFINITY;
            }
        };
        auto weigh = [&](f32x16 &t, const f32x16 &e, int from, int to) {
#pragma unroll
            for (int i = from; i < to; ++i) t[i] = __builtin_amdgcn_exp2f(fmaf(t[i], c, -base)) * (e[i] - delta);
        };
        auto gradient = [&](f32x16 &t, const f32x16 &e, uint32_t place) {
            RowsOperand<T> ds;
            weigh(t, e, 0, 16);
            ds.set(t);
            mma_rows<RB>(kt, place, ds, dq);
        };
        auto step = [&](f32x16 &t, f32x16 &e, f32x16 &nt, f32x16 &ne, int u, uint32_t next_at, uint32_t own_at) {
            fill.next();  // tiles u + 3: their places were last read in step u - 1
            if constexpr (sizeof(T) == 2) {
                // in the order it is to run: LDS reads ahead of their use, the arithmetic between the products
                constexpr int AHEAD = NJ < 2 ? NJ : 2;
                Raw16 k[NJ], v[NJ], r[2 * DB], ds[2];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    k[j] = lds_read16(ka.at[j] + next_at);
                    v[j] = lds_read16(ka.at[j] + next_at + V0);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (j + AHEAD < NJ) {
                        k[j + AHEAD] = lds_read16(ka.at[j + AHEAD] + next_at);
                        v[j + AHEAD] = lds_read16(ka.at[j + AHEAD] + next_at + V0);
                    } else if (j + AHEAD - NJ < 2 * DB) {
                        r[j + AHEAD - NJ] = rows_piece<RB>(kt, own_at, j + AHEAD - NJ);
                    }
                    nt = mma_pieces<T>(k[j], q[j], j ? nt : f32x16{});
                    weigh(t, e, 16 * j / NJ, 16 * j / NJ + 8 / NJ);
                    __builtin_amdgcn_sched_barrier(0);
                    ne = mma_pieces<T>(v[j], g[j], j ? ne : f32x16{});
                    weigh(t, e, 16 * j / NJ + 8 / NJ, 16 * (j + 1) / NJ);
                    __builtin_amdgcn_sched_barrier(0);
                }
                ds[0] = pack8(t, 0);
                ds[1] = pack8(t, 1);
#pragma unroll
                for (int x = 0; x < 2 * DB; ++x) {
                    if (x + AHEAD < 2 * DB) r[x + AHEAD] = rows_piece<RB>(kt, own_at, x + AHEAD);
                    dq[x % DB] = mma_pieces<T>(r[x], ds[x / DB], dq[x % DB]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                constexpr int AHEAD = NJ < 2 ? NJ : 2, FAR = 8;
                Raw16 k[NJ], v[NJ];
                float r[16 * DB];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    k[j] = lds_read16(ka.at[j] + next_at);
                    v[j] = lds_read16(ka.at[j] + next_at + V0);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (j + AHEAD < NJ) {
                        k[j + AHEAD] = lds_read16(ka.at[j + AHEAD] + next_at);
                        v[j + AHEAD] = lds_read16(ka.at[j + AHEAD] + next_at + V0);
                    } else {
#pragma unroll
                        for (int x = 0; x < FAR / AHEAD; ++x)
                            r[(j + AHEAD - NJ) * (FAR / AHEAD) + x] = rows_piece<RB>(kt, own_at, (j + AHEAD - NJ) * (FAR / AHEAD) + x);
                    }
                    nt = mma_pieces<T>(k[j], q[j], j ? nt : f32x16{});
                    ne = mma_pieces<T>(v[j], g[j], j ? ne : f32x16{});
                    weigh(t, e, 16 * j / NJ, 16 * (j + 1) / NJ);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int x = 0; x < 16 * DB; ++x) {
                    if (x + FAR < 16 * DB) r[x + FAR] = rows_piece<RB>(kt, own_at, x + FAR);
                    dq[x % DB] = __builtin_amdgcn_mfma_f32_32x32x2f32(r[x], t[x / DB], dq[x % DB], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            mask(nt, u + 1);
            wait_copies_and_barrier<PER>();
        };
        if (steps) {
            wait_copies_and_barrier<2 * PER>();
            products(s[0], dp[0], 0);
            mask(s[0], 0);
            wait_copies_and_barrier<PER>();
            int u = 0;
            for (; u + 2 < steps; u += 2) {  // ring places u mod 4 = 0 or 2: the addresses move to the other half
                const uint32_t other = u & 2 ? -2 * TILE : 2 * TILE;
                step(s[0], dp[0], s[1], dp[1], u, TILE, 0);
                ka.move(other);
                step(s[1], dp[1], s[0], dp[0], u + 1, 0, TILE);
                kt.move(other);
            }
            if (u + 1 < steps) {
                step(s[0], dp[0], s[1], dp[1], u, TILE, 0);
                gradient(s[1], dp[1], TILE);
            } else {
                gradient(s[0], dp[0], 0);
            }
            if (u & 2) {
                ka.move(-2 * TILE);
                kt.move(-2 * TILE);
            }
            wait_copies_and_barrier<0>();
        }
        if constexpr (SPLIT)
            store_rows<float>(dq, 1.0f, A.part + (split * A.nq * A.heads + at) * A.dim, A.dim, valid);
        else if (w.pieces > 1)
            store_rows<float>(dq, 1.0f, A.part + ((int64_t)w.index * BWD_ROWS + (threadIdx.x >> 6) * 32 + (lane & 31)) * A.dim, A.dim, valid);
        else
            store_rows<T>(dq, A.scale, (T *)A.dq.p + (q_beg + token) * A.dq.row + head * A.dq.head, A.dim, valid);
    }
}

// A step handles 32 query rows of the group: s = q k^T and dp = g v^T of the next rows
// are formed while p and ds of its own are computed, then dv^T += g^T p and dk^T += q^T ds.
// Rows past the end are copied as zeros; their scores and dp are 0 times a key's elements,
// which is not 0 where the key holds an infinity, so their weights are set to 0.
// Same rows: 755 us, 0.92 PFLOP/s of its four products.  At 128 elements a head the keys,
// values and both gradients take 192 registers, so one wave runs on a SIMD and its LDS
// reads and barriers are hidden only by its own products; in fp32 the next products'
// operands do not fit and 141 to 143 registers are spilled (8000 x 4 x 128: 2.64 ms, 99 TFLOP/s).
constexpr int dkv_residency(int rb) { return rb > 128 ? 1 : 2; }  // waves a SIMD

template <typename T, int DP, bool SPLIT, bool DIRECT>
__global__ __launch_bounds__(64 * BWD_WAVES, dkv_residency(DP * sizeof(T))) void k_attn_dkv(AttnArgs A)
{
    constexpr int RB = DP * (int)sizeof(T), NJ = RB / 32, DB = DP / 32, TILE = 32 * RB;
    constexpr uint32_t G0 = RING * TILE, STAT0 = 2 * RING * TILE;
    __shared__ __attribute__((aligned(1024))) char smem[2 * RING * TILE + RING * BWD_WAVES * 256];
    const uint32_t lds = (uint32_t)(uintptr_t)(SC_LDS char *)smem;

    const Ragged rq = {A.q_off, A.entries, A.nq, A.group}, rk = {A.k_off, A.entries, A.nk, 1};
    Work w;
    int64_t ktile, row0 = 0, split = 0;
    if constexpr (SPLIT) {
        if (!find_work(rq, rk, A.chunk, xcd_work(), A.kv_heads * A.tiles, 0, false, &w) || !w.real) return;
        split = w.tile;
        row0 = split * A.chunk;
        ktile = w.which % A.tiles;
        w.which /= A.tiles;
    } else {
        if (!find_work(rk, rq, BWD_ROWS, xcd_work(), A.kv_heads, A.slots, false, &w)) return;
        ktile = w.tile;
    }
    const int hk = (int)w.which;
    const int64_t q_beg = SPLIT ? w.own_beg : w.other_beg, k_beg = SPLIT ? w.other_beg : w.own_beg;
    const int64_t keys = SPLIT ? w.other_len : w.own_len;
    int64_t rows64 = (SPLIT ? w.own_len : w.other_len) * A.group - row0;
    if (SPLIT && rows64 <= 0) return;  // a number without a run (see first_tile)
    if (SPLIT && rows64 > A.chunk) rows64 = A.chunk;
    if (!SPLIT && w.pieces > 1) {
        piece_rows(w, w.other_len * A.group, &row0, &rows64);
        rows64 -= row0;
    }
    const int rows = (int)rows64, steps = (rows + 31) / 32;

    const int lane = lane_id(), half = lane >> 5, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const float c = A.scale * LOG2E;
    const uint32_t group = A.group;
    Fill<T, RB, BWD_WAVES, RING, DIRECT> fill;
    constexpr int PER = Fill<T, RB, BWD_WAVES, RING, DIRECT>::PER + 1;  // and the rows' statistics
    fill.init(lds, lds + G0, group == 1 ? A.q.row : 0, group == 1 ? A.grad.row : 0, A.dim);
    HeadAddr<RB> qa(lds);
    RowsAddr<T, RB> qt(lds);
    const uint32_t my_stat = lds + STAT0 + wave * 256;  // each wave keeps its own copy
    auto copy = [&](int a) {                            // the rows of step a: their places were last read in step a - 4
        const uint32_t first = (uint32_t)row0 + a * 32;
        const int left = rows - a * 32;
        // (base, delta) of 32 rows: one word a lane
        const uint32_t t0 = group == 1 ? first : first / group, r = first + lane / 2, t = group == 1 ? r : r / group;
        const float *sp = A.stat + ((q_beg + t0) * A.heads + hk * group) * 2;
        const uint32_t o = lane / 2 < left ? ((t - t0) * A.heads + (r - t * group)) * 8 + (lane & 1) * 4 : OUT_OF_RANGE;
        const uint32_t to = my_stat + (a & (RING - 1)) * (BWD_WAVES * 256);
        if constexpr (DIRECT) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(scalar_rsrc(sp, 0x7fffffff), (SC_LDS void *)(uintptr_t)__builtin_amdgcn_readfirstlane(to), 4, o, 0, 0, 0);
        } else {
            *(SC_LDS float *)(uintptr_t)(to + lane * 4) = o != OUT_OF_RANGE ? *(const float *)((const char *)sp + o) : 0.0f;
        }
        if (group == 1) fill.next();
        else fill.next_grouped(A.q, A.grad, q_beg, hk * group, first, group);
    };

    for (; ktile * BWD_ROWS < keys; ktile += SPLIT ? A.tiles : keys) {
        const int64_t wave_key = ktile * BWD_ROWS + wave * 32;
        if (SPLIT) __syncthreads();
        fill.start((const T *)A.q.p + (q_beg + row0) * A.q.row + hk * A.q.head,
                   (const T *)A.grad.p + (q_beg + row0) * A.grad.row + hk * A.grad.head, rows);  // (group = 1)
        if (steps)
            for (int u = 0; u < RING - 1; ++u) copy(u);
        if (wave_key >= keys) {
            if (steps) {
                wait_copies_and_barrier<2 * PER>();
                for (int u = 0; u < steps; ++u) {
                    if (u) copy(u + RING - 2);
                    wait_copies_and_barrier<PER>();
                }
                wait_copies_and_barrier<0>();
            }
            continue;
        }
        const int64_t key = wave_key + (lane & 31);
        const bool valid = key < keys;
        Raw16 k[NJ], v[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = (2 * j + half) * VEC<T>;
            k[j] = v[j] = Raw16{0, 0, 0, 0};
            if (valid && e < A.dim) {
                k[j] = *(const Raw16Any *)((const T *)A.k.p + (k_beg + key) * A.k.row + hk * A.k.head + e);
                v[j] = *(const Raw16Any *)((const T *)A.v.p + (k_beg + key) * A.v.row + hk * A.v.head + e);
            }
        }
        f32x16 dk[DB], dv[DB], s[2], dp[2];
#pragma unroll
        for (int db = 0; db < DB; ++db) dk[db] = dv[db] = f32x16{};
        auto products = [&](f32x16 &t, f32x16 &e, uint32_t place) {
            t = e = f32x16{};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                t = mma_pieces<T>(lds_read16(qa.at[j] + place), k[j], t);
                e = mma_pieces<T>(lds_read16(qa.at[j] + place + G0), v[j], e);
            }
        };
        // registers i, i + 1: rows 8 (i / 4) + 4 half + i % 4 and the next, two (base, delta) pairs
        auto stats = [&](int u, int i) {
            return __builtin_bit_cast(f32x4, lds_read16(my_stat + (u & (RING - 1)) * (BWD_WAVES * 256) + 32 * half + 64 * (i / 4) + 8 * (i % 4)));
        };
        auto weigh = [&](f32x16 &t, f32x16 &e, int i, f32x4 bd) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                t[i + x] = __builtin_amdgcn_exp2f(fmaf(t[i + x], c, -bd[2 * x]));
                e[i + x] = t[i + x] * (e[i + x] - bd[2 * x + 1]);
            }
        };
        // the last step, which alone has rows past the end
        auto gradient = [&](f32x16 &t, f32x16 &e, int u, uint32_t place) {
            RowsOperand<T> p, ds;
#pragma unroll
            for (int i = 0; i < 16; i += 2) weigh(t, e, i, stats(u, i));
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (8 * (i / 4) + 4 * half + i % 4 >= rows - u * 32) t[i] = e[i] = 0.0f;
            p.set(t);
            mma_rows<RB>(qt, place + G0, p, dv);
            ds.set(e);
            mma_rows<RB>(qt, place, ds, dk);
        };
        auto step = [&](f32x16 &t, f32x16 &e, f32x16 &nt, f32x16 &ne, int u, uint32_t next_at, uint32_t own_at) {
            copy(u + RING - 1);
            if constexpr (sizeof(T) == 2) {
                // in the order it is to run: LDS reads ahead of their use, the arithmetic between the products
                constexpr int AHEAD = NJ < 2 ? NJ : 2;
                Raw16 a[NJ], b[NJ], r[4 * DB], w[4];
                f32x4 bd[8];
                auto rows = [&](int x) { return rows_piece<RB>(qt, own_at + (x < 2 * DB ? G0 : 0), x % (2 * DB)); };
#pragma unroll
                for (int i = 0; i < 8; ++i) bd[i] = stats(u, 2 * i);
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    a[j] = lds_read16(qa.at[j] + next_at);
                    b[j] = lds_read16(qa.at[j] + next_at + G0);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (j + AHEAD < NJ) {
                        a[j + AHEAD] = lds_read16(qa.at[j + AHEAD] + next_at);
                        b[j + AHEAD] = lds_read16(qa.at[j + AHEAD] + next_at + G0);
                    } else {
                        r[2 * (j + AHEAD - NJ)] = rows(2 * (j + AHEAD - NJ));
                        r[2 * (j + AHEAD - NJ) + 1] = rows(2 * (j + AHEAD - NJ) + 1);
                    }
                    nt = mma_pieces<T>(a[j], k[j], j ? nt : f32x16{});
                    __builtin_amdgcn_sched_barrier(0);
                    ne = mma_pieces<T>(b[j], v[j], j ? ne : f32x16{});
#pragma unroll
                    for (int i = 8 * j / NJ; i < 8 * (j + 1) / NJ; ++i) weigh(t, e, 2 * i, bd[i]);
                    __builtin_amdgcn_sched_barrier(0);
                }
                w[0] = pack8(t, 0);
                w[1] = pack8(t, 1);
                w[2] = pack8(e, 0);
                w[3] = pack8(e, 1);
#pragma unroll
                for (int x = 0; x < 4 * DB; ++x) {
                    if (x + 2 * AHEAD < 4 * DB) r[x + 2 * AHEAD] = rows(x + 2 * AHEAD);
                    f32x16 &d = x < 2 * DB ? dv[x % DB] : dk[x % DB];
                    d = mma_pieces<T>(r[x], w[x / DB], d);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                constexpr int AHEAD = NJ < 2 ? NJ : 2, FAR = 8;
                Raw16 a[NJ], b[NJ];
                float r[32 * DB];
                f32x4 bd[8];
                auto rows = [&](int x) { return rows_piece<RB>(qt, own_at + (x < 16 * DB ? G0 : 0), x % (16 * DB)); };
#pragma unroll
                for (int i = 0; i < 8; ++i) bd[i] = stats(u, 2 * i);
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    a[j] = lds_read16(qa.at[j] + next_at);
                    b[j] = lds_read16(qa.at[j] + next_at + G0);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (j + AHEAD < NJ) {
                        a[j + AHEAD] = lds_read16(qa.at[j + AHEAD] + next_at);
                        b[j + AHEAD] = lds_read16(qa.at[j + AHEAD] + next_at + G0);
                    } else {
#pragma unroll
                        for (int x = 0; x < FAR / AHEAD; ++x)
                            r[(j + AHEAD - NJ) * (FAR / AHEAD) + x] = rows((j + AHEAD - NJ) * (FAR / AHEAD) + x);
                    }
                    nt = mma_pieces<T>(a[j], k[j], j ? nt : f32x16{});
                    ne = mma_pieces<T>(b[j], v[j], j ? ne : f32x16{});
#pragma unroll
                    for (int i = 8 * j / NJ; i < 8 * (j + 1) / NJ; ++i) weigh(t, e, 2 * i, bd[i]);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int x = 0; x < 32 * DB; ++x) {
                    if (x + FAR < 32 * DB) r[x + FAR] = rows(x + FAR);
                    const int y = x % (16 * DB);
                    f32x16 &d = x < 16 * DB ? dv[y % DB] : dk[y % DB];
                    d = __builtin_amdgcn_mfma_f32_32x32x2f32(r[x], x < 16 * DB ? t[y / DB] : e[y / DB], d, 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            wait_copies_and_barrier<PER>();
        };
        if (steps) {
            wait_copies_and_barrier<2 * PER>();
            products(s[0], dp[0], 0);
            wait_copies_and_barrier<PER>();
            int u = 0;
            for (; u + 2 < steps; u += 2) {
                const uint32_t other = u & 2 ? -2 * TILE : 2 * TILE;
                step(s[0], dp[0], s[1], dp[1], u, TILE, 0);
                qa.move(other);
                step(s[1], dp[1], s[0], dp[0], u + 1, 0, TILE);
                qt.move(other);
            }
            if (u + 1 < steps) {
                step(s[0], dp[0], s[1], dp[1], u, TILE, 0);
                gradient(s[1], dp[1], u + 1, TILE);
            } else {
                gradient(s[0], dp[0], u, 0);
            }
            if (u & 2) {
                qa.move(-2 * TILE);
                qt.move(-2 * TILE);
            }
            wait_copies_and_barrier<0>();
        }
        if constexpr (SPLIT) {
            const int64_t at = ((split * A.nk + k_beg + key) * A.kv_heads + hk) * A.dim;
            store_rows<float>(dk, 1.0f, A.part + at, A.dim, valid);
            store_rows<float>(dv, 1.0f, A.part2 + at, A.dim, valid);
        } else if (w.pieces > 1) {
            const int64_t at = ((int64_t)w.index * BWD_ROWS + wave * 32 + (lane & 31)) * A.dim;
            store_rows<float>(dk, 1.0f, A.part + at, A.dim, valid);
            store_rows<float>(dv, 1.0f, A.part2 + at, A.dim, valid);
        } else {
            store_rows<T>(dk, A.scale, (T *)A.dk.p + (k_beg + key) * A.dk.row + hk * A.dk.head, A.dim, valid);
            store_rows<T>(dv, 1.0f, (T *)A.dv.p + (k_beg + key) * A.dv.row + hk * A.dv.head, A.dim, valid);
        }
    }
}

// Every variant that is launched, spelled out: the host pass leaves some of them out when they
// are only named in a launch.
#define VARIANTS(T, DP, DIRECT) \
    template __global__ void k_attn_dq<T, DP, false, DIRECT>(AttnArgs); \
    template __global__ void k_attn_dq<T, DP, true, DIRECT>(AttnArgs); \
    template __global__ void k_attn_dkv<T, DP, false, DIRECT>(AttnArgs); \
    template __global__ void k_attn_dkv<T, DP, true, DIRECT>(AttnArgs);
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

// One wave to an output row: the splits' partial gradients of an [n, heads, dim] tensor
// summed in order of their number and scaled, for one or two such tensors (blockIdx.y).
// `other` is the side that was split.
constexpr int SUM_WAVES = 4;
template <typename T>
__global__ __launch_bounds__(64 * SUM_WAVES) void k_attn_sum(Ragged own, Ragged other, int heads, int dim, int chunk,
                                                             const float *__restrict__ part_a, float scale_a, Heads out_a,
                                                             const float *__restrict__ part_b, float scale_b, Heads out_b)
{
    __shared__ f32x4 acc[SUM_WAVES][64];
    const float *part = blockIdx.y ? part_b : part_a;
    const float scale = blockIdx.y ? scale_b : scale_a;
    const Heads out = blockIdx.y ? out_b : out_a;
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    const int64_t at = (int64_t)blockIdx.x * SUM_WAVES + wave, rows = own.n * heads;
    const bool on = at < rows;
    const int64_t row = on ? at / heads : 0;
    const int head = (int)(at - row * heads), p = find_part(own, row);
    const bool real = on && p >= 1 && p <= own.entries;
    const int64_t len = real ? (other.bound(p + 1) - other.bound(p)) * other.mult : 0;
    const int n = len > 0 ? (int)((len + chunk - 1) / chunk) : 0;
    const int pieces = dim / 4, groups = 64 / pieces, g = lane / pieces, e = lane % pieces;
    f32x4 sum = {0, 0, 0, 0};
    if (g < groups) {
#pragma unroll 8
        for (int s = g; s < n; s += groups) sum += *(const f32x4 *)(part + (s * rows + at) * dim + 4 * e);
    }
    acc[wave][lane] = sum;
    __syncthreads();
    if (!on || g) return;
    for (int i = 1; i < groups; ++i) sum += acc[wave][i * pieces + e];
    store4((T *)out.p + row * out.row + head * out.head + 4 * e, sum * scale);
}

// The pieces of cut tiles summed and scaled, for one or two tensors (blockIdx.z): blockIdx.x
// counts the tiles, blockIdx.y their quarters.  own: the side whose rows the tiles are.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_sum_cut(Ragged own, Ragged other, int kv_heads, int group, int dim, uint32_t slots,
                                                      const float *__restrict__ part_a, float scale_a, Heads out_a,
                                                      const float *__restrict__ part_b, float scale_b, Heads out_b)
{
    Work w;
    if (!find_work(own, other, BWD_ROWS, blockIdx.x, kv_heads, slots, true, &w)) return;
    const float *part = blockIdx.z ? part_b : part_a;
    const float scale = blockIdx.z ? scale_b : scale_a;
    const Heads out = blockIdx.z ? out_b : out_a;
    const int pieces = dim / 4, groups = 256 / pieces, g = threadIdx.x / pieces, e = threadIdx.x % pieces;
    const int64_t rows = w.own_len * group - w.tile * BWD_ROWS;
    if (g >= groups) return;
    for (int r = blockIdx.y * (BWD_ROWS / 4) + g; r < (int)(blockIdx.y + 1) * (BWD_ROWS / 4) && r < rows; r += groups) {
        const uint32_t row = (uint32_t)(w.tile * BWD_ROWS) + r, token = group == 1 ? row : row / group;
        const int head = (int)(w.which * group + (row - token * group));
        f32x4 v[MAX_PIECES];
#pragma unroll
        for (uint32_t i = 0; i < MAX_PIECES; ++i)
            v[i] = i < w.pieces ? *(const f32x4 *)(part + ((int64_t)(w.index + i) * BWD_ROWS + r) * dim + 4 * e) : f32x4{0, 0, 0, 0};
        f32x4 sum = v[0];
#pragma unroll
        for (uint32_t i = 1; i < MAX_PIECES; ++i) sum += v[i];
        store4((T *)out.p + (w.own_beg + token) * out.row + head * out.head + 4 * e, sum * scale);
    }
}

struct BwdPlan {
    SplitPlan q, k;
    uint32_t q_slots, k_slots;  // blocks that run at once where tiles may be cut
    size_t stat, part;  // bytes of the workspace's two areas
};

static BwdPlan bwd_plan(const AttnArgs &A, int dtype)
{
    const int rb = (A.dim + 31) / 32 * 32 * (dtype == SUBMCONV_F32 ? 4 : 2);
    BwdPlan p;
    const int q_slots = blocks_at_once(rb, dq_residency(rb)), k_slots = blocks_at_once(rb, dkv_residency(rb));
    p.q = split_plan(A.nq * A.group, BWD_ROWS, A.nk, 32, A.entries, A.kv_heads, q_slots, dtype);
    p.k = split_plan(A.nk, BWD_ROWS, A.nq * A.group, 32, A.entries, A.kv_heads, k_slots, dtype);
    p.q_slots = cut_pays(A.nk, A.entries, dtype) ? (uint32_t)q_slots : 0;
    p.k_slots = cut_pays(A.nq * A.group, A.entries, dtype) ? (uint32_t)k_slots : 0;
    p.stat = ((size_t)A.nq * A.heads * 2 * sizeof(float) + 15) / 16 * 16;
    const size_t row = A.dim * sizeof(float), tile = BWD_ROWS * row;
    const size_t a = p.q.chunk ? (size_t)p.q.splits * A.nq * A.heads * row : 2 * p.q_slots * tile;
    const size_t b = p.k.chunk ? (size_t)p.k.splits * A.nk * A.kv_heads * 2 * row : 4 * p.k_slots * tile;
    p.part = a > b ? a : b;  // the two passes use it one after the other
    return p;
}

size_t attention_backward_workspace(const AttnArgs &A, int dtype)
{
    const BwdPlan p = bwd_plan(A, dtype);
    return p.stat + p.part;
}

static void set_split(AttnArgs &A, const SplitPlan &p)
{
    A.chunk = p.chunk;
    A.tiles = p.tiles;
}

template <typename T, int DP, bool DIRECT>
static int run_bwd(AttnArgs A, const BwdPlan &p, hipStream_t st)
{
    const dim3 block(64 * BWD_WAVES);
    const Ragged rq = {A.q_off, A.entries, A.nq, 1}, rk = {A.k_off, A.entries, A.nk, 1};
    if (A.nq) {
        if (p.q.chunk) {
            set_split(A, p.q);
            const int64_t work = ragged_tiles(A.nk, A.entries, 1, A.chunk) * A.kv_heads * A.tiles;
            hipLaunchKernelGGL((k_attn_dq<T, DP, true, DIRECT>), dim3(xcd_grid(work)), block, 0, st, A);
            SC_LAUNCHED("attention_backward queries (split)");
            hipLaunchKernelGGL(k_attn_sum<T>, dim3((unsigned)((A.nq * A.heads + SUM_WAVES - 1) / SUM_WAVES)), dim3(64 * SUM_WAVES), 0, st, rq, rk, A.heads, A.dim,
                               A.chunk, A.part, A.scale, A.dq, nullptr, 0.0f, Heads{});
        } else {
            A.slots = DIRECT ? p.q_slots : 0;
            const int64_t work = ragged_tiles(A.nq, A.entries, A.group, BWD_ROWS) * A.kv_heads + 2 * A.slots;
            hipLaunchKernelGGL((k_attn_dq<T, DP, false, DIRECT>), dim3(xcd_grid(work)), block, 0, st, A);
            if (A.slots) {
                SC_LAUNCHED("attention_backward queries");
                const Ragged own = {A.q_off, A.entries, A.nq, A.group};
                hipLaunchKernelGGL(k_attn_sum_cut<T>, dim3(A.slots, 4), dim3(256), 0, st, own, rk, A.kv_heads, A.group, A.dim, A.slots,
                                   A.part, A.scale, A.dq, nullptr, 0.0f, Heads{});
            }
        }
        SC_LAUNCHED("attention_backward queries");
    }
    if (A.nk) {
        if (p.k.chunk) {
            set_split(A, p.k);
            A.part2 = A.part + p.k.splits * A.nk * A.kv_heads * A.dim;
            const int64_t work = ragged_tiles(A.nq, A.entries, A.group, A.chunk) * A.kv_heads * A.tiles;
            hipLaunchKernelGGL((k_attn_dkv<T, DP, true, DIRECT>), dim3(xcd_grid(work)), block, 0, st, A);
            SC_LAUNCHED("attention_backward keys (split)");
            const Ragged rows = {A.q_off, A.entries, A.nq, A.group};
            hipLaunchKernelGGL(k_attn_sum<T>, dim3((unsigned)((A.nk * A.kv_heads + SUM_WAVES - 1) / SUM_WAVES), 2), dim3(64 * SUM_WAVES), 0, st, rk, rows, A.kv_heads,
                               A.dim, A.chunk, A.part, A.scale, A.dk, A.part2, 1.0f, A.dv);
        } else {
            A.slots = DIRECT ? p.k_slots : 0;
            A.part2 = A.part + (size_t)2 * A.slots * BWD_ROWS * A.dim;
            const int64_t work = ragged_tiles(A.nk, A.entries, 1, BWD_ROWS) * A.kv_heads + 2 * A.slots;
            hipLaunchKernelGGL((k_attn_dkv<T, DP, false, DIRECT>), dim3(xcd_grid(work)), block, 0, st, A);
            if (A.slots) {
                SC_LAUNCHED("attention_backward keys");
                const Ragged other = {A.q_off, A.entries, A.nq, A.group};
                hipLaunchKernelGGL(k_attn_sum_cut<T>, dim3(A.slots, 4, 2), dim3(256), 0, st, rk, other, A.kv_heads, 1, A.dim, A.slots,
                                   A.part, A.scale, A.dk, A.part2, 1.0f, A.dv);
            }
        }
        SC_LAUNCHED("attention_backward keys");
    }
    return SUBMCONV_OK;
}

// Whether all tiles can be copied straight into LDS (see Fill).
static bool direct(const AttnArgs &A, int es)
{
    uintptr_t bits = 0;
    for (const Heads *h : {&A.q, &A.k, &A.v, &A.grad}) bits |= (uintptr_t)h->p | (uintptr_t)(h->row * es) | (uintptr_t)(h->head * es);
    const int64_t far = (A.q.head > A.grad.head ? A.q.head : A.grad.head) * A.group * es;  // heads of a group
    return !(bits & 15) && A.k.row >= A.dim && A.v.row >= A.dim &&
           (A.group == 1 ? A.q.row >= A.dim && A.grad.row >= A.dim : far < int64_t(1) << 30);
}

int attention_backward(AttnArgs A, int dtype, void *workspace, hipStream_t st)
{
    const BwdPlan p = bwd_plan(A, dtype);
    A.stat = (float *)workspace;
    A.part = (float *)((char *)workspace + p.stat);
    const int dp = (A.dim + 31) / 32;
#define GO(T)                                                                  \
    if (!direct(A, sizeof(T))) return run_bwd<T, 128, false>(A, p, st);        \
    switch (dp) {                                                              \
    case 1: return run_bwd<T, 32, true>(A, p, st);                             \
    case 2: return run_bwd<T, 64, true>(A, p, st);                             \
    case 3: return run_bwd<T, 96, true>(A, p, st);                             \
    default: return run_bwd<T, 128, true>(A, p, st);                           \
    }
    if (dtype == SUBMCONV_F32) {
        GO(float)
    } else {
        GO(uint16_t)
    }
#undef GO
}

}  // namespace sc
