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

constexpr int BWD_WAVES = 4, BWD_ROWS = 32 * BWD_WAVES;
template <typename T> constexpr int BWD_TILE = sizeof(T) == 2 ? 64 : 32;

// A score's exponent is s c - base; a query whose scores are all -inf has lse = -inf and
// weights exp(-inf), so its base must be finite.
__device__ __forceinline__ float lse_base(float lse) { return lse == -INFINITY ? 0.0f : lse * LOG2E; }

template <typename T, int DP, bool SPLIT>
__global__ __launch_bounds__(64 * BWD_WAVES, DP <= 64 ? 2 : 1) void k_attn_dq(AttnArgs A)
{
    constexpr int RB = DP * (int)sizeof(T), NJ = RB / 32, DB = DP / 32, KT = BWD_TILE<T>, KB = KT / 32;
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
        const int64_t slots = A.nq * A.group / BWD_ROWS + A.entries + 2, w = xcd_work();
        if (w >= slots * A.kv_heads) return;
        hk = (int)(w / slots);
        find_tile(rq, BWD_ROWS, w % slots, &part, &qtile);
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

    for (; qtile * BWD_ROWS < rows; qtile += SPLIT ? A.tiles : rows) {
        const int64_t wave_row = qtile * BWD_ROWS + (threadIdx.x >> 6) * 32;
        const bool busy = wave_row < rows;
        const uint32_t row = (uint32_t)(wave_row + (lane & 31));
        const bool valid = row < rows;
        const uint32_t token = A.group == 1 ? row : row / A.group, head = hk * A.group + (row - token * A.group);
        const int64_t at = (q_beg + token) * A.heads + head;
        Raw16 q[NJ], g[NJ];
        float base = 0.0f, delta = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) q[j] = g[j] = Raw16{0, 0, 0, 0};
        if (valid) {
            const T *qp = (const T *)A.q.p + (q_beg + token) * A.q.row + head * A.q.head;
            const T *gp = (const T *)A.grad.p + (q_beg + token) * A.grad.row + head * A.grad.head;
            const T *op = (const T *)A.out.p + (q_beg + token) * A.out.row + head * A.out.head;
            base = lse_base(A.lse[at]);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int e = (2 * j + half) * VEC<T>;
                if (e >= A.dim) continue;
                q[j] = *(const Raw16Any *)(qp + e);
                g[j] = *(const Raw16Any *)(gp + e);
                float a[VEC<T>], b[VEC<T>];
                unpack(g[j], a, gp);
                unpack((Raw16) * (const Raw16Any *)(op + e), b, gp);
#pragma unroll
                for (int i = 0; i < VEC<T>; ++i) delta += a[i] * b[i];
            }
        }
        delta += other_half(delta);
        if (valid && half == 0 && split == 0) A.delta[at] = delta;

        f32x16 dq[DB];
#pragma unroll
        for (int db = 0; db < DB; ++db) dq[db] = f32x16{};
        TileLoad<T, RB, KT, 64 * BWD_WAVES> tk, tv;
        HeadAddr<RB> ka(lds);
        RowsAddr<T, RB> kt(lds);
        if (SPLIT) __syncthreads();
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
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    f32x16 s = {}, dp = {};
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        s = mma_pieces<T>(lds_read16(ka.at[j] + buf + kb * 32 * RB), q[j], s);
                        dp = mma_pieces<T>(lds_read16(ka.at[j] + buf + TILE + kb * 32 * RB), g[j], dp);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (left < KT && kb * 32 + 8 * (i / 4) + 4 * half + i % 4 >= left) s[i] = -INFINITY;
                        s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -base)) * (dp[i] - delta);
                    }
                    RowsOperand<T> ds;
                    ds.set(s);
                    mma_rows<RB>(kt, buf + kb * 32 * RB, ds, dq);
                }
            }
            if (left > KT) {
                tk.store(lds + (buf ^ BUF));
                tv.store(lds + (buf ^ BUF) + TILE);
            }
            __syncthreads();
        }
        if (!busy) continue;
        if constexpr (SPLIT)
            store_rows<float>(dq, 1.0f, A.part + (split * A.nq * A.heads + at) * A.dim, A.dim, valid);
        else
            store_rows<T>(dq, A.scale, (T *)A.dq.p + (q_beg + token) * A.dq.row + head * A.dq.head, A.dim, valid);
    }
}

template <typename T, int DP, bool SPLIT>
__global__ __launch_bounds__(64 * BWD_WAVES, DP <= 64 ? 2 : 1) void k_attn_dkv(AttnArgs A)
{
    constexpr int RB = DP * (int)sizeof(T), NJ = RB / 32, DB = DP / 32, QT = BWD_TILE<T>, QB = QT / 32;
    constexpr int TILE = QT * RB, BUF = 2 * TILE;
    __shared__ __attribute__((aligned(16))) char smem[2 * BUF];
    __shared__ __attribute__((aligned(16))) float stat[2][2][QT];  // base and delta of a tile's queries
    const uint32_t lds = (uint32_t)(uintptr_t)(SC_LDS char *)smem;

    const Ragged rq = {A.q_off, A.entries, A.nq, A.group}, rk = {A.k_off, A.entries, A.nk, 1};
    int part, hk;
    int64_t ktile, row0 = 0, split = 0;
    if constexpr (SPLIT) {
        const int64_t slots = A.nq * A.group / A.chunk + A.entries + 2, w = xcd_work();
        if (w >= slots * A.kv_heads * A.tiles) return;
        hk = (int)(w / (slots * A.tiles));
        ktile = w / slots % A.tiles;
        find_tile(rq, A.chunk, w % slots, &part, &split);
        row0 = split * A.chunk;
    } else {
        const int64_t slots = A.nk / BWD_ROWS + A.entries + 2, w = xcd_work();
        if (w >= slots * A.kv_heads) return;
        hk = (int)(w / slots);
        find_tile(rk, BWD_ROWS, w % slots, &part, &ktile);
    }
    const int64_t q_beg = rq.bound(part), k_beg = rk.bound(part);
    const bool real = part >= 1 && part <= A.entries;
    const int64_t keys = rk.bound(part + 1) - k_beg;
    int64_t rows = real ? (rq.bound(part + 1) - q_beg) * A.group - row0 : 0;
    if (SPLIT && (rows <= 0 || !real)) return;
    if (SPLIT && rows > A.chunk) rows = A.chunk;
    if (rows < 0) rows = 0;

    const int lane = lane_id(), half = lane >> 5;
    const float c = A.scale * LOG2E;
    const T *qp = (const T *)A.q.p + q_beg * A.q.row + (int64_t)hk * A.group * A.q.head;
    const T *gp = (const T *)A.grad.p + q_beg * A.grad.row + (int64_t)hk * A.group * A.grad.head;

    for (; ktile * BWD_ROWS < keys; ktile += SPLIT ? A.tiles : keys) {
        const int64_t wave_key = ktile * BWD_ROWS + (threadIdx.x >> 6) * 32;
        const bool busy = wave_key < keys;
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
        f32x16 dk[DB], dv[DB];
#pragma unroll
        for (int db = 0; db < DB; ++db) dk[db] = dv[db] = f32x16{};
        TileLoad<T, RB, QT, 64 * BWD_WAVES> tq, tg;
        HeadAddr<RB> qa(lds);
        RowsAddr<T, RB> qt(lds);
        float nb = 0.0f, nd = 0.0f;
        auto fetch = [&](int64_t r0) {  // rows past the run weigh exp(-inf)
            const int n = (int)(rows - r0 < QT ? rows - r0 : QT);
            tq.load_grouped(qp, A.q.row, A.q.head, (uint32_t)(row0 + r0), A.group, n, A.dim);
            tg.load_grouped(gp, A.grad.row, A.grad.head, (uint32_t)(row0 + r0), A.group, n, A.dim);
            if (threadIdx.x < QT) {
                nb = INFINITY;
                nd = 0.0f;
                if ((int)threadIdx.x < n) {
                    const uint32_t r = (uint32_t)(row0 + r0) + threadIdx.x, token = A.group == 1 ? r : r / A.group;
                    const int64_t at = (q_beg + token) * A.heads + hk * A.group + (r - token * A.group);
                    nb = lse_base(A.lse[at]);
                    nd = A.delta[at];
                }
            }
        };
        auto put = [&](uint32_t to, int b) {
            tq.store(lds + to);
            tg.store(lds + to + TILE);
            if (threadIdx.x < QT) {
                stat[b][0][threadIdx.x] = nb;
                stat[b][1][threadIdx.x] = nd;
            }
        };
        if (SPLIT) __syncthreads();
        if (rows > 0) {
            fetch(0);
            put(0, 0);
        }
        __syncthreads();
        uint32_t buf = 0;
        for (int64_t r0 = 0; r0 < rows; r0 += QT, buf ^= BUF) {
            const bool more = rows - r0 > QT;
            if (more) fetch(r0 + QT);
            if (busy) {
                const float *st = &stat[buf ? 1 : 0][0][0];
#pragma unroll
                for (int qb = 0; qb < QB; ++qb) {
                    f32x16 s = {}, dp = {};
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        s = mma_pieces<T>(lds_read16(qa.at[j] + buf + qb * 32 * RB), k[j], s);
                        dp = mma_pieces<T>(lds_read16(qa.at[j] + buf + TILE + qb * 32 * RB), v[j], dp);
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const f32x4 b = *(const f32x4 *)(st + qb * 32 + 2 * i + 4 * half);
                        const f32x4 d = *(const f32x4 *)(st + QT + qb * 32 + 2 * i + 4 * half);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            s[i + x] = __builtin_amdgcn_exp2f(fmaf(s[i + x], c, -b[x]));
                            dp[i + x] = s[i + x] * (dp[i + x] - d[x]);
                        }
                    }
                    RowsOperand<T> p, ds;
                    p.set(s);
                    mma_rows<RB>(qt, buf + TILE + qb * 32 * RB, p, dv);
                    ds.set(dp);
                    mma_rows<RB>(qt, buf + qb * 32 * RB, ds, dk);
                }
            }
            if (more) put(buf ^ BUF, buf ? 0 : 1);
            __syncthreads();
        }
        if (!busy) continue;
        if constexpr (SPLIT) {
            const int64_t at = ((split * A.nk + k_beg + key) * A.kv_heads + hk) * A.dim;
            store_rows<float>(dk, 1.0f, A.part + at, A.dim, valid);
            store_rows<float>(dv, 1.0f, A.part2 + at, A.dim, valid);
        } else {
            store_rows<T>(dk, A.scale, (T *)A.dk.p + (k_beg + key) * A.dk.row + hk * A.dk.head, A.dim, valid);
            store_rows<T>(dv, 1.0f, (T *)A.dv.p + (k_beg + key) * A.dv.row + hk * A.dv.head, A.dim, valid);
        }
    }
}

// One block to an output row: the splits' partial gradients of an [n, heads, dim] tensor
// summed in order of their number and scaled.  `other` is the side that was split.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_sum(Ragged own, Ragged other, int heads, int dim, int chunk,
                                                  const float *__restrict__ part, float scale, Heads out)
{
    __shared__ f32x4 acc[256];
    const int64_t at = blockIdx.x, row = at / heads;
    const int head = (int)(at - row * heads), p = find_part(own, row);
    const bool real = p >= 1 && p <= own.entries;
    const int64_t len = real ? (other.bound(p + 1) - other.bound(p)) * other.mult : 0;
    const int n = len > 0 ? (int)((len + chunk - 1) / chunk) : 0;
    const int pieces = dim / 4, groups = 256 / pieces, g = threadIdx.x / pieces, e = threadIdx.x % pieces;
    f32x4 sum = {0, 0, 0, 0};
    if (g < groups)
        for (int s = g; s < n; s += groups) sum += *(const f32x4 *)(part + (s * own.n * heads + at) * dim + 4 * e);
    acc[threadIdx.x] = sum;
    __syncthreads();
    if (g == 0) {
        for (int i = 1; i < groups; ++i) sum += acc[i * pieces + e];
        sum *= scale;
        T *op = (T *)out.p + row * out.row + head * out.head + 4 * e;
        if constexpr (sizeof(T) == 2) {
            const uint32_t a = pack_bf16(sum[0], sum[1]), b = pack_bf16(sum[2], sum[3]);
            op[0] = (uint16_t)a;
            op[1] = (uint16_t)(a >> 16);
            op[2] = (uint16_t)b;
            op[3] = (uint16_t)(b >> 16);
        } else {
            *(Raw16Any *)op = __builtin_bit_cast(Raw16, sum);
        }
    }
}

struct BwdPlan {
    SplitPlan q, k;
    size_t delta, part;  // bytes of the workspace's two areas
};

static BwdPlan bwd_plan(const AttnArgs &A, int dtype)
{
    const int tile = dtype == SUBMCONV_F32 ? BWD_TILE<float> : BWD_TILE<uint16_t>;
    BwdPlan p;
    p.q = split_plan(A.nq * A.group, BWD_ROWS, A.nk, tile, A.entries, A.kv_heads);
    p.k = split_plan(A.nk, BWD_ROWS, A.nq * A.group, tile, A.entries, A.kv_heads);
    p.delta = ((size_t)A.nq * A.heads * sizeof(float) + 15) / 16 * 16;
    const size_t a = p.q.chunk ? (size_t)p.q.splits * A.nq * A.heads * A.dim * sizeof(float) : 0;
    const size_t b = p.k.chunk ? (size_t)p.k.splits * A.nk * A.kv_heads * A.dim * 2 * sizeof(float) : 0;
    p.part = a > b ? a : b;  // the two passes use it one after the other
    return p;
}

size_t attention_backward_workspace(const AttnArgs &A, int dtype)
{
    const BwdPlan p = bwd_plan(A, dtype);
    return p.delta + p.part;
}

static void set_split(AttnArgs &A, const SplitPlan &p)
{
    A.chunk = p.chunk;
    A.splits = p.splits;
    A.tiles = p.tiles;
}

template <typename T, int DP>
static int run_bwd(AttnArgs A, const BwdPlan &p, hipStream_t st)
{
    const dim3 block(64 * BWD_WAVES);
    const Ragged rq = {A.q_off, A.entries, A.nq, 1}, rk = {A.k_off, A.entries, A.nk, 1};
    if (A.nq) {
        if (p.q.chunk) {
            set_split(A, p.q);
            const int64_t work = ragged_tiles(A.nk, A.entries, 1, A.chunk) * A.kv_heads * A.tiles;
            hipLaunchKernelGGL((k_attn_dq<T, DP, true>), dim3(xcd_grid(work)), block, 0, st, A);
            SC_LAUNCHED("attention_backward queries (split)");
            hipLaunchKernelGGL(k_attn_sum<T>, dim3((unsigned)(A.nq * A.heads)), dim3(256), 0, st, rq, rk, A.heads, A.dim,
                               A.chunk, A.part, A.scale, A.dq);
        } else {
            const int64_t work = ragged_tiles(A.nq, A.entries, A.group, BWD_ROWS) * A.kv_heads;
            hipLaunchKernelGGL((k_attn_dq<T, DP, false>), dim3(xcd_grid(work)), block, 0, st, A);
        }
        SC_LAUNCHED("attention_backward queries");
    }
    if (A.nk) {
        if (p.k.chunk) {
            set_split(A, p.k);
            A.part2 = A.part + p.k.splits * A.nk * A.kv_heads * A.dim;
            const int64_t work = ragged_tiles(A.nq, A.entries, A.group, A.chunk) * A.kv_heads * A.tiles;
            hipLaunchKernelGGL((k_attn_dkv<T, DP, true>), dim3(xcd_grid(work)), block, 0, st, A);
            SC_LAUNCHED("attention_backward keys (split)");
            const Ragged rows = {A.q_off, A.entries, A.nq, A.group};
            const dim3 grid((unsigned)(A.nk * A.kv_heads));
            hipLaunchKernelGGL(k_attn_sum<T>, grid, dim3(256), 0, st, rk, rows, A.kv_heads, A.dim, A.chunk, A.part,
                               A.scale, A.dk);
            hipLaunchKernelGGL(k_attn_sum<T>, grid, dim3(256), 0, st, rk, rows, A.kv_heads, A.dim, A.chunk, A.part2,
                               1.0f, A.dv);
        } else {
            const int64_t work = ragged_tiles(A.nk, A.entries, 1, BWD_ROWS) * A.kv_heads;
            hipLaunchKernelGGL((k_attn_dkv<T, DP, false>), dim3(xcd_grid(work)), block, 0, st, A);
        }
        SC_LAUNCHED("attention_backward keys");
    }
    return SUBMCONV_OK;
}

int attention_backward(AttnArgs A, int dtype, void *workspace, hipStream_t st)
{
    const BwdPlan p = bwd_plan(A, dtype);
    A.delta = (float *)workspace;
    A.part = (float *)((char *)workspace + p.delta);
    const int dp = (A.dim + 31) / 32;
#define GO(T)                                   \
    switch (dp) {                               \
    case 1: return run_bwd<T, 32>(A, p, st);    \
    case 2: return run_bwd<T, 64>(A, p, st);    \
    case 3: return run_bwd<T, 96>(A, p, st);    \
    default: return run_bwd<T, 128>(A, p, st);  \
    }
    if (dtype == SUBMCONV_F32) {
        GO(float)
    } else {
        GO(uint16_t)
    }
#undef GO
}

}  // namespace sc
