// The sum of a row's expert results, weighted by its gates, and its gradients:
//
//   out[n] = sum_j gate[n,j] y[slot[n,j]],   dy[slot[n,j]] = gate[n,j] g[n],   dgate[n,j] = g[n] . y[slot[n,j]]
//
// Sums are fp32 in the order of j.  Bound by memory: y is read once and out written once (backward:
// g and y read, dy written), 16 bytes a lane; a row's slots and gates are a few words that its
// lanes share.  Rows of y come in any order, a whole row at a time.  Measured in bf16: forward 1,187,403 x 2 of 64
// 84 us (5.7 TB/s), 20,384 x 4 of 1024 37 us (5.7; a copy reaches 4.9); backward 63 us for the latter, 6.0 TB/s (y from the
// forward pass is still in the memory-side cache).
#include "rowvec.h"

namespace sc {

constexpr int64_t COMBINE_BLOCKS = 1 << 22;  // along x (a launch's axis holds 2^32 threads); the rest along y

// A thread owns one piece of 16 bytes of a row (blocks of whole rows), all k loads in flight for
// K of them at a time.
template <typename T, int K>
__global__ __launch_bounds__(256) void k_combine(const T *__restrict__ y, int64_t ldy, int64_t np, const int32_t *__restrict__ slots,
                                                 const float *__restrict__ gates, int64_t n, int k, int c, int pieces, int rows_per_block,
                                                 T *__restrict__ out, int64_t ldo)
{
    constexpr int V = VEC<T>;
    const int r = pieces < 256 ? threadIdx.x / pieces : 0;
    const int64_t row = ((int64_t)blockIdx.y * COMBINE_BLOCKS + blockIdx.x) * rows_per_block + r;
    if (r >= rows_per_block || row >= n) return;
    for (int piece = threadIdx.x - r * pieces; piece < pieces; piece += 256) {
        const int e = piece * V, nv = c - e < V ? c - e : V;
        float sum[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = 0.0f;
        for (int j0 = 0; j0 < k; j0 += K) {
            Raw16 v[K];
            float f[K];
            bool on[K];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                const int64_t at = j0 + j < k ? slots[row * k + j0 + j] : -1;
                on[j] = at >= 0 && at < np;
                f[j] = on[j] && gates ? gates[row * k + j0 + j] : 1.0f;
                if (on[j]) v[j] = load_raw(y + at * ldy + e, nv);
            }
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (!on[j]) continue;
                float t[V];
                unpack(v[j], t, y);
#pragma unroll
                for (int i = 0; i < V; ++i) sum[i] += f[j] * t[i];
            }
        }
        store_raw(out + row * ldo + e, repack(sum, y), nv);
    }
}

// TPR threads walk a row; K: most slots a row has.  A row of dy is written by the pair that
// owns it: the first slot of row rows[p] that is p; its gate is the sum over that row's slots that are p.
// Rows of dy without an owner become zeros.
template <typename T, int K, int TPR>
__global__ __launch_bounds__(256) void k_combine_bwd(const T *__restrict__ g, int64_t ldg, const T *__restrict__ y, int64_t ldy, int64_t np,
                                                     const int32_t *__restrict__ slots, const int32_t *__restrict__ rows,
                                                     const float *__restrict__ gates, int64_t n, int k, int c, T *__restrict__ dy,
                                                     int64_t lddy, float *__restrict__ dgates)
{
    constexpr int V = VEC<T>, RPB = 256 / TPR;
    __shared__ float part[4][K];
    const int t = threadIdx.x % TPR, q = threadIdx.x / TPR, pieces = (c + V - 1) / V;
    const int64_t step = (int64_t)gridDim.x * RPB;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < n; row0 += step) {
        const int64_t row = row0 + q;
        const bool on = row < n;
        int64_t at[K];
        float f[K], dot[K];
        bool mine[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            at[j] = on && j < k ? slots[row * k + j] : -1;
            if (at[j] < 0 || at[j] >= np) at[j] = -1;
            f[j] = at[j] >= 0 && gates ? gates[row * k + j] : 1.0f;
            mine[j] = dy && at[j] >= 0 && rows[at[j]] == row;
            dot[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < j; ++i)
                if (mine[i] && at[i] == at[j]) {  // the same place twice in a row: its owner takes both gates
                    f[i] += f[j];
                    mine[j] = false;
                }
        for (int piece = t; piece < pieces; piece += TPR) {
            if (!on) break;
            const int e = piece * V, nv = c - e < V ? c - e : V;
            float gv[V];
            unpack(load_raw(g + row * ldg + e, nv), gv, g);
            Raw16 v[K];
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (dgates && at[j] >= 0) v[j] = load_raw(y + at[j] * ldy + e, nv);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (dgates && at[j] >= 0) {
                    float yv[V];
                    unpack(v[j], yv, g);
#pragma unroll
                    for (int i = 0; i < V; ++i) dot[j] += gv[i] * yv[i];
                }
                if (mine[j]) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = f[j] * gv[i];
                    store_raw(dy + at[j] * lddy + e, repack(o, g), nv);
                }
            }
        }
        if (dgates) {
#pragma unroll
            for (int j = 0; j < K; ++j) dot[j] = lanes_sum<(TPR < 64 ? TPR : 64)>(dot[j]);
            if constexpr (TPR > 64) {
                __syncthreads();
                if ((threadIdx.x & 63) == 0)
#pragma unroll
                    for (int j = 0; j < K; ++j) part[threadIdx.x >> 6][j] = dot[j];
                __syncthreads();
#pragma unroll
                for (int j = 0; j < K; ++j) dot[j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
            }
            if (on && t == 0)
                for (int j = 0; j < K; ++j)
                    if (j < k) dgates[row * k + j] = dot[j];
        }
    }
    if (!dy) return;
    // 64 places at a time: those that no row owns become zeros
    const int lane = threadIdx.x & 63;
    for (int64_t p0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 64; p0 < np; p0 += (int64_t)gridDim.x * 256) {
        bool lost = false;
        if (p0 + lane < np) {
            const int64_t r = rows[p0 + lane];
            lost = true;
            if (r >= 0 && r < n)
                for (int j = 0; j < k; ++j) lost = lost && slots[r * k + j] != p0 + lane;
        }
        for (uint64_t m = __ballot(lost); m; m &= m - 1) {
            T *to = dy + (p0 + __builtin_ctzll(m)) * lddy;
            for (int piece = lane; piece < pieces; piece += 64) store_raw(to + piece * V, Raw16{0, 0, 0, 0}, c - piece * V < V ? c - piece * V : V);
        }
    }
}

int combine(const void *y, int64_t ldy, int64_t np, const int32_t *slots, const float *gates, int64_t n, int k, int c, int dtype, void *out,
            int64_t ldo, hipStream_t st)
{
    const int v = dtype == SUBMCONV_F32 ? 4 : 8, pieces = (c + v - 1) / v, rows = pieces < 256 ? 256 / pieces : 1;
    const int64_t blocks = (n + rows - 1) / rows;
    const dim3 grid((unsigned)(blocks < COMBINE_BLOCKS ? blocks : COMBINE_BLOCKS), (unsigned)((blocks + COMBINE_BLOCKS - 1) / COMBINE_BLOCKS));
#define GO(T, K) hipLaunchKernelGGL((k_combine<T, K>), grid, dim3(256), 0, st, (const T *)y, ldy, np, slots, gates, n, k, c, pieces, rows, (T *)out, ldo)
#define BY_K(T) if (k == 1) GO(T, 1); else if (k == 2) GO(T, 2); else GO(T, 4)
    if (dtype == SUBMCONV_F32) { BY_K(float); } else { BY_K(uint16_t); }
#undef BY_K
#undef GO
    SC_LAUNCHED("combine");
    return SUBMCONV_OK;
}

int combine_backward(const void *g, int64_t ldg, const void *y, int64_t ldy, int64_t np, const int32_t *slots, const int32_t *rows,
                     const float *gates, int64_t n, int k, int c, int dtype, void *dy, int64_t lddy, float *dgates, hipStream_t st)
{
    const int v = dtype == SUBMCONV_F32 ? 4 : 8, pieces = (c + v - 1) / v;
    const int tpr = pieces <= 8 ? 8 : (pieces <= 128 ? 64 : 256);
    const int64_t a = (n + 256 / tpr - 1) / (256 / tpr), b = (np + 255) / 256, blocks = a > b ? a : b;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
#define GO(T, K, TPR)                                                                                                                  \
    hipLaunchKernelGGL((k_combine_bwd<T, K, TPR>), grid, dim3(256), 0, st, (const T *)g, ldg, (const T *)y, ldy, np, slots, rows, gates, n, k, c, \
                       (T *)dy, lddy, dgates)
#define BY_TPR(T, K) if (tpr == 8) GO(T, K, 8); else if (tpr == 64) GO(T, K, 64); else GO(T, K, 256)
#define BY_K(T) if (k <= 1) { BY_TPR(T, 1); } else if (k <= 2) { BY_TPR(T, 2); } else if (k <= 4) { BY_TPR(T, 4); } else if (k <= 8) { BY_TPR(T, 8); } else { BY_TPR(T, 16); }
    if (dtype == SUBMCONV_F32) { BY_K(float) } else { BY_K(uint16_t) }
#undef BY_K
#undef BY_TPR
#undef GO
    SC_LAUNCHED("combine_backward");
    return SUBMCONV_OK;
}

}  // namespace sc
