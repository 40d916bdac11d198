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
// values in LDS, two buffers, the next tile's loads in flight during the products.
#include "attention.h"

namespace sc {

// What a row's running maximum may be passed by, in powers of two, before the sums are
// rescaled: weights stay below 2^8, far from overflow, and most tiles skip the rescaling.
constexpr float SLACK = 8.0f;

// A weight is exp2(s c - m c) with c = scale log2(e) and m the row's running maximum: one
// fused rounding of the difference, and the rounding of m c is a common factor of a row's
// weights and their sum.  Past this size of m c that factor could overflow (and m c
// itself); the weight is then exp2((s - m) c), where equal scores cancel exactly.
constexpr float HUGE_BASE = 1073741824.0f;
__device__ __forceinline__ bool huge(float m, float c) { return m != -INFINITY && !(fabsf(m * c) <= HUGE_BASE); }

// What sums relative to the maximum m are worth relative to next >= m.
__device__ __forceinline__ float rescale(float m, float next, float c)
{
    if (next == -INFINITY) return 1.0f;
    return __builtin_amdgcn_exp2f(huge(next, c) ? (m - next) * c : m * c - next * c);
}

// log sum exp from the maximum and the sum of the weights.
__device__ __forceinline__ float log_sum(float m, float l, float scale)
{
    if (l == 0.0f) return -INFINITY;  // no key, or none with a finite score
    const float c = scale * LOG2E, e = __builtin_amdgcn_logf(l);
    return huge(m, c) ? m * scale + e * LN2 : (m * c + e) * LN2;
}

constexpr int FWD_WAVES = 4, FWD_ROWS = 32 * FWD_WAVES;
template <typename T> constexpr int FWD_KEYS = sizeof(T) == 2 ? 64 : 32;

// SPLIT: a block takes one run of `chunk` keys of an entry and leaves (sum, m, l) of it
// in part / part2 for k_attn_join; otherwise a block takes one tile of query rows over
// all keys.
template <typename T, int DP, bool SPLIT>
__global__ __launch_bounds__(64 * FWD_WAVES, 2) void k_attn(AttnArgs A)
{
    constexpr int RB = DP * (int)sizeof(T), NJ = RB / 32, DB = DP / 32, KT = FWD_KEYS<T>, KB = KT / 32;
    constexpr int TILE = KT * RB, BUF = 2 * TILE;
    __shared__ __attribute__((aligned(16))) char smem[2 * BUF];
    const uint32_t lds = (uint32_t)(uintptr_t)(SC_LDS char *)smem;

    const Ragged rq = {A.q_off, A.entries, A.nq, A.group}, rk = {A.k_off, A.entries, A.nk, 1};
    int part, hk;
    int64_t qtile, key0 = 0, split = 0;
    if constexpr (SPLIT) {
        const int64_t slots = A.nk / A.chunk + A.entries + 2, w = xcd_work();
        if (w >= slots * A.kv_heads * A.tiles) return;
        hk = (int)(w / (slots * A.tiles));
        qtile = w / slots % A.tiles;
        find_tile(rk, A.chunk, w % slots, &part, &split);
        key0 = split * A.chunk;
    } else {
        const int64_t slots = A.nq * A.group / FWD_ROWS + A.entries + 2, w = xcd_work();
        if (w >= slots * A.kv_heads) return;
        hk = (int)(w / slots);
        find_tile(rq, FWD_ROWS, w % slots, &part, &qtile);
    }
    const int64_t q_beg = rq.bound(part), k_beg = rk.bound(part);
    const bool real = part >= 1 && part <= A.entries;
    const int64_t rows = (rq.bound(part + 1) - q_beg) * A.group;
    int64_t keys = real ? rk.bound(part + 1) - k_beg - key0 : 0;
    if (SPLIT && (keys <= 0 || !real)) return;
    if (SPLIT && keys > A.chunk) keys = A.chunk;
    if (keys < 0) keys = 0;

    const int lane = lane_id(), half = lane >> 5;
    const float c = A.scale * LOG2E;
    const T *kp = (const T *)A.k.p + (k_beg + key0) * A.k.row + hk * A.k.head;
    const T *vp = (const T *)A.v.p + (k_beg + key0) * A.v.row + hk * A.v.head;

    for (; qtile * FWD_ROWS < rows; qtile += SPLIT ? A.tiles : rows) {
        const int64_t wave_row = qtile * FWD_ROWS + (threadIdx.x >> 6) * 32;
        const bool busy = wave_row < rows;  // a wave past the entry's rows only helps with the tiles
        const uint32_t row = (uint32_t)(wave_row + (lane & 31));
        const bool valid = row < rows;
        const uint32_t token = A.group == 1 ? row : row / A.group, head = hk * A.group + (row - token * A.group);
        Raw16 q[NJ];
        {
            const T *qp = (const T *)A.q.p + (q_beg + (valid ? token : 0)) * A.q.row + (valid ? head : 0) * A.q.head;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int e = (2 * j + half) * VEC<T>;
                q[j] = Raw16{0, 0, 0, 0};
                if (valid && e < A.dim) q[j] = *(const Raw16Any *)(qp + e);
            }
        }
        f32x16 o[DB];
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] = f32x16{};
        float m = -INFINITY, l = 0.0f;

        TileLoad<T, RB, KT, 64 * FWD_WAVES> tk, tv;
        HeadAddr<RB> ka(lds);
        RowsAddr<T, RB> va(lds + TILE);
        if (SPLIT) __syncthreads();  // the last tile's readers are done before it is written again
        if (keys > 0) {
            tk.load(kp, A.k.row, (int)(keys < KT ? keys : KT), A.dim);
            tv.load(vp, A.v.row, (int)(keys < KT ? keys : KT), A.dim);
            tk.store(lds);
            tv.store(lds + TILE);
        }
        __syncthreads();
        uint32_t buf = 0;
        for (int64_t k0 = 0; k0 < keys; k0 += KT, buf ^= BUF) {
            const int64_t left = keys - k0;
            if (left > KT) {
                const int n = (int)(left - KT < KT ? left - KT : KT);
                tk.load(kp + (k0 + KT) * A.k.row, A.k.row, n, A.dim);
                tv.load(vp + (k0 + KT) * A.v.row, A.v.row, n, A.dim);
            }
            if (busy) {
                f32x16 s[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    s[kb] = f32x16{};
#pragma unroll
                    for (int j = 0; j < NJ; ++j) s[kb] = mma_pieces<T>(lds_read16(ka.at[j] + buf + kb * 32 * RB), q[j], s[kb]);
                }
                if (left < KT) {
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (kb * 32 + 8 * (i / 4) + 4 * half + i % 4 >= left) s[kb][i] = -INFINITY;
                }
                float top = s[0][0];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kb][i]);
                top = fmaxf(top, other_half(top));
                if (__ballot((top - m) * c > SLACK)) {
                    const float next = fmaxf(m, top), f = rescale(m, next, c);
                    m = next;
                    l *= f;
#pragma unroll
                    for (int db = 0; db < DB; ++db) o[db] *= f;
                }
                float base = m == -INFINITY ? 0.0f : m * c, cs = c;  // no finite score yet: weights are exp(-inf)
                if (__ballot(huge(m, c))) {
                    const bool mine = huge(m, c);
                    cs = 1.0f;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; ++i) s[kb][i] = mine ? (s[kb][i] - m) * c : fmaf(s[kb][i], c, -base);
                    base = 0.0f;
                }
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        s[kb][i] = __builtin_amdgcn_exp2f(fmaf(s[kb][i], cs, -base));
                        l += s[kb][i];
                    }
                    RowsOperand<T> p;
                    p.set(s[kb]);
                    mma_rows<RB>(va, buf + kb * 32 * RB, p, o);
                }
            }
            if (left > KT) {
                tk.store(lds + (buf ^ BUF));
                tv.store(lds + (buf ^ BUF) + TILE);
            }
            __syncthreads();
        }
        if (!busy) continue;
        l += other_half(l);
        if constexpr (SPLIT) {
            const int64_t at = split * A.nq * A.heads + (q_beg + token) * A.heads + head;
            store_rows<float>(o, 1.0f, A.part + at * A.dim, A.dim, valid);
            if (valid && half == 0) *(float2 *)(A.part2 + 2 * at) = make_float2(m, l);
        } else {
            T *op = (T *)A.out.p + (q_beg + token) * A.out.row + head * A.out.head;
            store_rows<T>(o, l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l), op, A.dim, valid);
            if (A.lse && valid && half == 0)
                A.lse[(q_beg + token) * A.heads + head] = log_sum(m, l, A.scale);
        }
    }
}

// One block to a query row: the splits' sums joined in order of their number.
constexpr int JOIN_MAX_SPLITS = 2048;
template <typename T>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs A)
{
    __shared__ float w[JOIN_MAX_SPLITS];
    __shared__ float red[4];
    __shared__ f32x4 acc[256];
    const int64_t at = blockIdx.x, token = at / A.heads;
    const int head = (int)(at - token * A.heads);
    const Ragged rq = {A.q_off, A.entries, A.nq, 1}, rk = {A.k_off, A.entries, A.nk, 1};
    const int part = find_part(rq, token);
    const bool real = part >= 1 && part <= A.entries;
    const int64_t keys = real ? rk.bound(part + 1) - rk.bound(part) : 0;
    const int n = keys > 0 ? (int)((keys + A.chunk - 1) / A.chunk) : 0;
    const int64_t rows = A.nq * A.heads;
    const float c = A.scale * LOG2E;

    float top = -INFINITY;
    for (int s = threadIdx.x; s < n; s += 256) top = fmaxf(top, A.part2[2 * (s * rows + at)]);
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    float l = 0.0f;
    for (int s = threadIdx.x; s < n; s += 256) {
        const float2 ml = *(const float2 *)(A.part2 + 2 * (s * rows + at));
        const float f = rescale(ml.x, top, c);
        w[s] = f;
        l += ml.y * f;
    }
    l = lanes_sum<64>(l);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = l;
    __syncthreads();
    l = (red[0] + red[1]) + (red[2] + red[3]);

    const int pieces = A.dim / 4, groups = 256 / pieces, g = threadIdx.x / pieces, e = threadIdx.x % pieces;
    f32x4 sum = {0, 0, 0, 0};
    if (g < groups)
        for (int s = g; s < n; s += groups) sum += *(const f32x4 *)(A.part + (s * rows + at) * A.dim + 4 * e) * w[s];
    acc[threadIdx.x] = sum;
    __syncthreads();
    if (g == 0) {
        for (int i = 1; i < groups; ++i) sum += acc[i * pieces + e];
        sum *= l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        T *op = (T *)A.out.p + token * A.out.row + head * A.out.head + 4 * e;
        if constexpr (sizeof(T) == 2) {
            const uint32_t a = pack_bf16(sum[0], sum[1]), b = pack_bf16(sum[2], sum[3]);
            op[0] = (uint16_t)a;
            op[1] = (uint16_t)(a >> 16);
            op[2] = (uint16_t)b;
            op[3] = (uint16_t)(b >> 16);
        } else {
            *(Raw16Any *)op = __builtin_bit_cast(Raw16, sum);
        }
        if (A.lse && e == 0) A.lse[at] = log_sum(top, l, A.scale);
    }
}

// How a pass over a long side is split when its own side has few tiles: enough runs that
// all blocks together fill the card, none shorter than MIN_CHUNK rows.  chunk = 0: not at all.
constexpr int64_t WANT_BLOCKS = 768, MIN_CHUNK = 256;

SplitPlan split_plan(int64_t own_rows, int own_tile, int64_t other_rows, int other_tile, int entries, int kv_heads)
{
    SplitPlan p = {0, 0, 1};
    if (own_rows == 0 || other_rows == 0) return p;
    const int64_t per_entry = (own_rows / entries + own_tile - 1) / own_tile;
    const int64_t tiles = per_entry > 0 ? per_entry : 1;
    const int64_t used = entries < own_rows ? entries : own_rows;
    if (tiles * used * kv_heads * 2 > WANT_BLOCKS) return p;
    int64_t runs = WANT_BLOCKS / (tiles * kv_heads);
    if (runs > JOIN_MAX_SPLITS - 1) runs = JOIN_MAX_SPLITS - 1;
    int64_t chunk = (other_rows + runs - 1) / runs;
    if (chunk < MIN_CHUNK) chunk = MIN_CHUNK;
    chunk = (chunk + other_tile - 1) / other_tile * other_tile;
    if (chunk * 2 > other_rows / entries || chunk > (1 << 30)) return p;  // entries of one run or two: nothing to gain
    p.chunk = (int)chunk;
    p.splits = (other_rows + chunk - 1) / chunk;
    p.tiles = (int)tiles;
    return p;
}

static SplitPlan fwd_plan(const AttnArgs &A, int dtype)
{
    return split_plan(A.nq * A.group, FWD_ROWS, A.nk, dtype == SUBMCONV_F32 ? FWD_KEYS<float> : FWD_KEYS<uint16_t>,
                      A.entries, A.kv_heads);
}

size_t attention_workspace(const AttnArgs &A, int dtype)
{
    const SplitPlan p = fwd_plan(A, dtype);
    return p.chunk ? (size_t)p.splits * A.nq * A.heads * (A.dim + 2) * sizeof(float) : 0;
}

template <typename T, int DP>
static int run_fwd(AttnArgs A, const SplitPlan &p, void *workspace, hipStream_t st)
{
    if (p.chunk) {
        A.chunk = p.chunk;
        A.splits = p.splits;
        A.tiles = p.tiles;
        A.part = (float *)workspace;
        A.part2 = A.part + p.splits * A.nq * A.heads * A.dim;
        const int64_t work = ragged_tiles(A.nk, A.entries, 1, p.chunk) * A.kv_heads * p.tiles;
        hipLaunchKernelGGL((k_attn<T, DP, true>), dim3(xcd_grid(work)), dim3(64 * FWD_WAVES), 0, st, A);
        SC_LAUNCHED("attention (split)");
        hipLaunchKernelGGL((k_attn_join<T>), dim3((unsigned)(A.nq * A.heads)), dim3(256), 0, st, A);
        SC_LAUNCHED("attention join");
        return SUBMCONV_OK;
    }
    const int64_t work = ragged_tiles(A.nq, A.entries, A.group, FWD_ROWS) * A.kv_heads;
    hipLaunchKernelGGL((k_attn<T, DP, false>), dim3(xcd_grid(work)), dim3(64 * FWD_WAVES), 0, st, A);
    SC_LAUNCHED("attention");
    return SUBMCONV_OK;
}

int attention(const AttnArgs &A, int dtype, void *workspace, hipStream_t st)
{
    const SplitPlan p = fwd_plan(A, dtype);
    const int dp = (A.dim + 31) / 32;
#define GO(T)                                                \
    switch (dp) {                                            \
    case 1: return run_fwd<T, 32>(A, p, workspace, st);      \
    case 2: return run_fwd<T, 64>(A, p, workspace, st);      \
    case 3: return run_fwd<T, 96>(A, p, workspace, st);      \
    default: return run_fwd<T, 128>(A, p, workspace, st);    \
    }
    if (dtype == SUBMCONV_F32) {
        GO(float)
    } else {
        GO(uint16_t)
    }
#undef GO
}

}  // namespace sc
