// The k best experts of each row, their gates, and the plan that groups the (row, expert) pairs by
// expert; the gradient of the scores.
//
// Order of a row's scores: descending, equal ones by number; a NaN comes before all else; -inf is
// a closed expert and is never taken.  Gates are exp(v_j - v_0) over their sum (over the chosen
// ones, or over all experts), in fp32.
//
// The plan: pair row * k + j of an expert stands behind the pairs of earlier experts and those
// of the same expert in earlier rows (a stable counting sort); pairs without an expert come last.
//   k_route_top    a block's rows: experts and gates, and how many pairs each expert gets
//   k_route_scan   for each expert, where each block's pairs begin among the expert's
//   k_route_place  a block's pairs to their places, in order
// All counts are whole numbers, so the plan does not depend on the order of atomics.  Each kernel
// is bound by memory where rows are many (the scores are read once), and by its launch where few.
#include "rowvec.h"

namespace sc {

constexpr int ROUTE_PAIRS = 2048;  // pairs of a block, about

// A score's order as a whole number: larger is better; NaN above all, -0 like +0, the lowest
// value is for what may not be taken (again).
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
constexpr uint32_t KEY_CLOSED = 0x007fffffu;  // of -inf
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k == 0xffffffffu ? 0x7fc00000u : (k >> 31 ? k ^ 0x80000000u : ~k));
}

// Of two (key, number) pairs the better one: larger key, then smaller number.
struct Best {
    uint32_t key, number;
};
__device__ __forceinline__ Best better(Best a, Best b)
{
    return a.key > b.key || (a.key == b.key && a.number < b.number) ? a : b;
}
template <int L>
__device__ __forceinline__ Best lanes_best(Best b)
{
#pragma unroll
    for (int o = 1; o < L; o <<= 1) b = better(b, Best{(uint32_t)__shfl_xor((int)b.key, o, 64), (uint32_t)__shfl_xor((int)b.number, o, 64)});
    return b;
}

// L lanes hold a row's scores, CH pieces of 16 bytes each.
template <typename T, int L, int CH>
__global__ __launch_bounds__(256) void k_route_top(const T *__restrict__ logits, int64_t ld, int64_t n, int experts, int k,
                                                   int normalize, int rows_per_block, int32_t *__restrict__ chosen,
                                                   float *__restrict__ gates, uint32_t *__restrict__ counts)
{
    constexpr int V = VEC<T>, RPB = 256 / L;
    __shared__ uint32_t hist[SUBMCONV_ROUTE_MAX_EXPERTS + 1];
    for (int i = threadIdx.x; i <= experts; i += 256) hist[i] = 0;
    __syncthreads();
    const int lane = threadIdx.x % L, g = threadIdx.x / L;
    const int64_t first = (int64_t)blockIdx.x * rows_per_block;
    const int64_t end = first + rows_per_block < n ? first + rows_per_block : n;
    for (int64_t row0 = first; row0 < end; row0 += RPB) {
        const int64_t row = row0 + g < end ? row0 + g : end - 1;
        const bool on = row0 + g < end;
        uint32_t key[CH][V];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int e = (i * L + lane) * V, nv = experts - e < 0 ? 0 : (experts - e < V ? experts - e : V);
            float v[V];
            unpack(load_raw(logits + row * ld + (nv ? e : 0), nv), v, logits);
#pragma unroll
            for (int j = 0; j < V; ++j) key[i][j] = j < nv ? order_key(v[j]) : 0;
        }
        float top = 0.0f, total = 0.0f;
        for (int j = 0; j < k; ++j) {
            Best b = {0, 0xffffffffu};
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) b = better(b, Best{key[i][q], (uint32_t)((i * L + lane) * V + q)});
            b = lanes_best<L>(b);
            const bool there = b.key > KEY_CLOSED;
            const float value = key_value(b.key);
            if (j == 0) {
                top = there ? value : 0.0f;
                if (!normalize) {
#pragma unroll
                    for (int i = 0; i < CH; ++i)
#pragma unroll
                        for (int q = 0; q < V; ++q)
                            if (key[i][q] > KEY_CLOSED) total += expf(key_value(key[i][q]) - top);
                    total = lanes_sum<L>(total);
                }
            }
            const float e = there ? expf(value - top) : 0.0f;
            if (normalize) total += e;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    if (b.number == (uint32_t)((i * L + lane) * V + q)) key[i][q] = 0;
            if (on && lane == 0) {
                const int32_t expert = there ? (int32_t)b.number : -1;
                chosen[row * k + j] = expert;
                gates[row * k + j] = e;  // divided below
                atomicAdd(&hist[there ? expert : experts], 1u);
            }
        }
        if (on && lane == 0)
            for (int j = 0; j < k; ++j) gates[row * k + j] = total == 0.0f ? 0.0f : gates[row * k + j] / total;
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= experts; i += 256) counts[(int64_t)i * gridDim.x + blockIdx.x] = hist[i];
}

// counts [bins][blocks] become, for each bin, exclusive sums over the blocks; totals [bins].
__global__ __launch_bounds__(256) void k_route_scan(uint32_t *__restrict__ counts, int blocks, uint32_t *__restrict__ totals)
{
    __shared__ uint32_t lds[4];
    uint32_t *mine = counts + (int64_t)blockIdx.x * blocks;
    uint32_t before = 0;
    for (int b0 = 0; b0 < blocks; b0 += 256) {
        const int b = b0 + threadIdx.x;
        const uint32_t v = b < blocks ? mine[b] : 0;
        uint32_t sum;
        const uint32_t incl = block_incl_scan256(v, lds, &sum);
        if (b < blocks) mine[b] = before + incl - v;
        before += sum;
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = before;
}

// The places of a block's pairs.  A wave takes a run of the block's pairs: it counts them by
// expert, the counts of the block's waves give each wave its first places, and 64 pairs at a
// time find their order among those of the same expert by comparing digits across the wave.
__global__ __launch_bounds__(256) void k_route_place(const int32_t *__restrict__ chosen, int64_t pairs, int k, int experts, int bits,
                                                     int pairs_per_block, const uint32_t *__restrict__ counts,
                                                     const uint32_t *__restrict__ totals, int32_t *__restrict__ offsets,
                                                     int32_t *__restrict__ rows, int32_t *__restrict__ slots)
{
    __shared__ uint32_t at[4][SUBMCONV_ROUTE_MAX_EXPERTS + 1];
    __shared__ uint32_t lds[4];
    const int bins = experts + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int i = threadIdx.x; i < 4 * (SUBMCONV_ROUTE_MAX_EXPERTS + 1); i += 256) (&at[0][0])[i] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * pairs_per_block;
    const int64_t end = first + pairs_per_block < pairs ? first + pairs_per_block : pairs;
    const int run = (pairs_per_block / 4 + 63) / 64 * 64;  // pairs of a wave
    const int64_t w0 = first + (int64_t)wave * run, w1 = w0 + run < end ? w0 + run : end;
    for (int64_t p = w0 + lane; p < w1; p += 64) {
        const int32_t e = chosen[p];
        atomicAdd(&at[wave][e < 0 ? experts : e], 1u);
    }
    __syncthreads();
    // bins in turns of 256: the place of each bin's first pair, then of each wave's
    uint32_t before = 0;
    for (int i0 = 0; i0 < bins; i0 += 256) {
        const int i = i0 + threadIdx.x;
        const uint32_t v = i < bins ? totals[i] : 0;
        uint32_t sum;
        const uint32_t start = before + block_incl_scan256(v, lds, &sum) - v;
        before += sum;
        if (i < bins) {
            if (blockIdx.x == 0) offsets[i] = (int32_t)start;  // offsets[experts]: where the pairs without an expert begin
            uint32_t place = start + counts[(int64_t)i * gridDim.x + blockIdx.x];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t c = at[w][i];
                at[w][i] = place;
                place += c;
            }
        }
    }
    __syncthreads();
    for (int64_t p0 = w0; p0 < w1; p0 += 64) {
        const int64_t p = p0 + lane;
        const bool on = p < w1;
        const int32_t c = on ? chosen[p] : 0;
        const uint32_t e = c < 0 ? experts : c;
        const uint64_t same = match_digit(e, on, bits);
        uint32_t place = 0;
        if (on) place = at[wave][e] + __popcll(same & lanemask_lt());
        // all lanes have read before the last of each expert moves its place on
        __builtin_amdgcn_wave_barrier();
        if (on && (same >> lane) == 1) at[wave][e] = place + 1;
        __builtin_amdgcn_wave_barrier();
        if (on) {
            slots[p] = (int32_t)place;
            rows[place] = (int32_t)(p / k);
        }
    }
}

// dL/dscore of expert e: with d_j = dgate_j gate_j,  [e = expert j] d_j - p_e sum(d)  where p is the
// softmax over the chosen experts or over all.
template <typename T, int L, int CH>
__global__ __launch_bounds__(256) void k_route_bwd(const float *__restrict__ grad, const T *__restrict__ logits, int64_t ld, int64_t n,
                                                   int experts, int k, int normalize, const int32_t *__restrict__ chosen,
                                                   const float *__restrict__ gates, T *__restrict__ out, int64_t out_ld)
{
    constexpr int V = VEC<T>, RPB = 256 / L;
    const int lane = threadIdx.x % L, g = threadIdx.x / L;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < n; row0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = row0 + g < n ? row0 + g : n - 1;
        const bool on = row0 + g < n;
        float v[CH][V];
        int nv[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int e = (i * L + lane) * V;
            nv[i] = experts - e < 0 ? 0 : (experts - e < V ? experts - e : V);
#pragma unroll
            for (int q = 0; q < V; ++q) v[i][q] = 0.0f;
            if (!normalize) unpack(load_raw(logits + row * ld + (nv[i] ? e : 0), nv[i]), v[i], out);
        }
        float sum = 0.0f;
        for (int j = 0; j < k; ++j) sum += grad[row * k + j] * gates[row * k + j];
        if (!normalize) {
            float top = -INFINITY, total = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    if (q < nv[i]) top = fmaxf(top, v[i][q]);
#pragma unroll
            for (int o = 1; o < L; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
            const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    v[i][q] = q < nv[i] ? expf(v[i][q] - from) : 0.0f;
                    total += v[i][q];
                }
            total = lanes_sum<L>(total);
            const float f = top == -INFINITY ? 0.0f : -sum / total;  // a row that is closed altogether has no gradient
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) v[i][q] *= f;
        }
        for (int j = 0; j < k; ++j) {
            const int32_t e = chosen[row * k + j];
            const float gate = gates[row * k + j];
            const float d = gate * (normalize ? grad[row * k + j] - sum : grad[row * k + j]);
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    if (e == (i * L + lane) * V + q) v[i][q] += d;
        }
        if (on) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (nv[i]) store_raw(out + row * out_ld + (i * L + lane) * V, repack(v[i], out), nv[i]);
        }
    }
}

// Lanes a row takes: a power of two with one or two pieces a lane.
#define ROUTE_LANES(K, T, ...)                                                                  \
    switch (lanes * 4 + ch) {                                                                   \
    case 1 * 4 + 1: hipLaunchKernelGGL((K<T, 1, 1>), grid, dim3(256), 0, st, __VA_ARGS__); break; \
    case 2 * 4 + 1: hipLaunchKernelGGL((K<T, 2, 1>), grid, dim3(256), 0, st, __VA_ARGS__); break; \
    case 4 * 4 + 1: hipLaunchKernelGGL((K<T, 4, 1>), grid, dim3(256), 0, st, __VA_ARGS__); break; \
    case 8 * 4 + 1: hipLaunchKernelGGL((K<T, 8, 1>), grid, dim3(256), 0, st, __VA_ARGS__); break; \
    case 16 * 4 + 1: hipLaunchKernelGGL((K<T, 16, 1>), grid, dim3(256), 0, st, __VA_ARGS__); break; \
    case 32 * 4 + 1: hipLaunchKernelGGL((K<T, 32, 1>), grid, dim3(256), 0, st, __VA_ARGS__); break; \
    case 64 * 4 + 1: hipLaunchKernelGGL((K<T, 64, 1>), grid, dim3(256), 0, st, __VA_ARGS__); break; \
    default:                                                                                    \
        if constexpr (sizeof(T) == 4) hipLaunchKernelGGL((K<T, 64, 2>), grid, dim3(256), 0, st, __VA_ARGS__); \
    }

static void route_shape(int experts, int dtype, int *lanes, int *ch)
{
    const int v = dtype == SUBMCONV_F32 ? 4 : 8, pieces = (experts + v - 1) / v;
    *lanes = 1;
    while (*lanes < pieces && *lanes < 64) *lanes *= 2;
    *ch = pieces > 64 ? 2 : 1;
}

static int route_rows(int k) { return ROUTE_PAIRS / k; }
static int64_t route_blocks(int64_t n, int k) { return (n + route_rows(k) - 1) / route_rows(k); }

size_t route_workspace(int64_t n, int experts, int k)
{
    return n ? (size_t)(route_blocks(n, k) + 1) * (experts + 1) * sizeof(uint32_t) : 0;
}

int route(const void *logits, int64_t ld, int64_t n, int experts, int k, int dtype, int normalize, int32_t *chosen, float *gates,
          int32_t *offsets, int32_t *rows, int32_t *slots, void *workspace, hipStream_t st)
{
    int lanes, ch;
    route_shape(experts, dtype, &lanes, &ch);
    const int64_t blocks = route_blocks(n, k);
    uint32_t *counts = (uint32_t *)workspace, *totals = counts + blocks * (experts + 1);
    const dim3 grid((unsigned)blocks);
    if (dtype == SUBMCONV_F32) {
        ROUTE_LANES(k_route_top, float, (const float *)logits, ld, n, experts, k, normalize, route_rows(k), chosen, gates, counts)
    } else {
        ROUTE_LANES(k_route_top, uint16_t, (const uint16_t *)logits, ld, n, experts, k, normalize, route_rows(k), chosen, gates, counts)
    }
    SC_LAUNCHED("route");
    hipLaunchKernelGGL(k_route_scan, dim3(experts + 1), dim3(256), 0, st, counts, (int)blocks, totals);
    SC_LAUNCHED("route sums");
    hipLaunchKernelGGL(k_route_place, grid, dim3(256), 0, st, chosen, n * k, k, experts, bits_for(experts + 1), route_rows(k) * k, counts,
                       totals, offsets, rows, slots);
    SC_LAUNCHED("route places");
    return SUBMCONV_OK;
}

// No rows: only the offsets are there to be written.
__global__ void k_route_none(int32_t *offsets, int many)
{
    for (int i = threadIdx.x; i < many; i += 256) offsets[i] = 0;
}
int route_none(int32_t *offsets, int experts, hipStream_t st)
{
    hipLaunchKernelGGL(k_route_none, dim3(1), dim3(256), 0, st, offsets, experts + 1);
    SC_LAUNCHED("route");
    return SUBMCONV_OK;
}

int route_backward(const float *grad, const void *logits, int64_t ld, int64_t n, int experts, int k, int dtype, int normalize,
                   const int32_t *chosen, const float *gates, void *out, int64_t out_ld, hipStream_t st)
{
    int lanes, ch;
    route_shape(experts, dtype, &lanes, &ch);
    const int64_t rpb = 256 / lanes, blocks = (n + rpb - 1) / rpb;
    const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
    if (dtype == SUBMCONV_F32) {
        ROUTE_LANES(k_route_bwd, float, grad, (const float *)logits, ld, n, experts, k, normalize, chosen, gates, (float *)out, out_ld)
    } else {
        ROUTE_LANES(k_route_bwd, uint16_t, grad, (const uint16_t *)logits, ld, n, experts, k, normalize, chosen, gates, (uint16_t *)out, out_ld)
    }
    SC_LAUNCHED("route_backward");
    return SUBMCONV_OK;
}

}  // namespace sc
