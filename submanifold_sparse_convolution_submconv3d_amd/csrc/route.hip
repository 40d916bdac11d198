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
// (few pairs: the first kernel alone; up to 64 blocks: without the second)
// All counts are whole numbers, so the plan does not depend on the order of atomics.  Each kernel
// is bound by its launches where rows are few (450 x 8 fp32, k = 2: one kernel, 9 us), by memory and instructions where
// many.  1,187,403 x 64 fp32, k = 4: top 108 us, scan 8, place 32, backward 122, where reading the scores once takes 62
// and reading them and writing their gradient 123 at the rate of a copy: the backward pass is at it, the top k is bound by
// the instructions of its sorting, and the scan by the latency of one block's walk for each expert.
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

// exp(d) for d <= 0, to a few roundings of d and of the result (the argument in units of log 2 is one
// rounding of d, the instruction one of the result); below the smallest normal number it is 0.  For the forward pass, which
// instructions bound; the backward pass, which memory bounds, has expf, and its p may differ from a gate in the last bits.
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * 1.4426950408889634f); }

// Larger of the group's keys, in every lane of aligned groups of L lanes (a power of two).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
    return v > o ? v : o;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    if constexpr (L >= 2) v = dpp_max<0xb1>(v);    // the steps of lanes_sum
    if constexpr (L >= 4) v = dpp_max<0x4e>(v);
    if constexpr (L >= 8) v = dpp_max<0x141>(v);
    if constexpr (L >= 16) v = dpp_max<0x140>(v);
    if constexpr (L >= 32) {
        auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = r[0] > r[1] ? r[0] : r[1];
    }
    if constexpr (L >= 64) {
        auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = r[0] > r[1] ? r[0] : r[1];
    }
    return v;
}

// What the wave's lanes wrote to LDS is read by the others from here on.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Where a block's pairs go.  A wave takes a run of `WAVE_PAIRS` of them, 64 at a time: they find their
// order among those of the same expert by comparing digits across the wave, and a count of the
// wave's pairs of each expert so far.  The counts of the block's waves then give each wave its first
// places.  at [4][experts + 1] and lds [4] are LDS.  BASE(bin) is where the block's pairs of a bin begin
// among all of the bin's, TOTAL(bin) how many the bin has.
constexpr int WAVE_CHUNKS = ROUTE_PAIRS / 4 / 64;
template <class Base, class Total>
__device__ __forceinline__ void place_pairs(const int32_t *chosen, int64_t first, int64_t end, int k, int experts, int bits,
                                            uint32_t (*at)[SUBMCONV_ROUTE_MAX_EXPERTS + 1], uint32_t *lds, Base base, Total total,
                                            int32_t *offsets, int32_t *rows, int32_t *slots)
{
    const int bins = experts + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int i = threadIdx.x; i < bins; i += 256)
#pragma unroll
        for (int w = 0; w < 4; ++w) at[w][i] = 0;
    const int64_t w0 = first + (int64_t)wave * (WAVE_CHUNKS * 64);
    int32_t e[WAVE_CHUNKS];
    uint32_t in_wave[WAVE_CHUNKS];
#pragma unroll
    for (int c = 0; c < WAVE_CHUNKS; ++c) {
        const int64_t p = w0 + c * 64 + lane;
        const int32_t v = p < end ? chosen[p] : 0;
        e[c] = v < 0 ? experts : v;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < WAVE_CHUNKS; ++c) {
        const bool on = w0 + c * 64 + lane < end;
        const uint64_t same = match_digit((uint32_t)e[c], on, bits);
        in_wave[c] = 0;
        if (on) in_wave[c] = at[wave][e[c]] + __popcll(same & lanemask_lt());
        // all lanes have read before the last of each expert moves its count on
        wave_sync();
        if (on && (same >> lane) == 1) at[wave][e[c]] = in_wave[c] + 1;
        wave_sync();
    }
    __syncthreads();
    uint32_t before = 0;
    for (int i0 = 0; i0 < bins; i0 += 256) {
        const int i = i0 + threadIdx.x;
        const uint32_t v = i < bins ? total(i) : 0;
        uint32_t sum;
        const uint32_t start = before + block_incl_scan256(v, lds, &sum) - v;
        before += sum;
        if (i < bins) {
            if (first == 0) offsets[i] = (int32_t)start;  // offsets[experts]: where the pairs without an expert begin
            uint32_t place = start + base(i);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t c = at[w][i];
                at[w][i] = place;
                place += c;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < WAVE_CHUNKS; ++c) {
        const int64_t p = w0 + c * 64 + lane;
        if (p >= end) continue;
        const uint32_t place = at[wave][e[c]] + in_wave[c];
        slots[p] = (int32_t)place;
        rows[place] = (int32_t)(p / k);
    }
}

// L lanes hold a row's scores, 16 neighbouring ones each.  A lane first sorts the K (>= k) best of its own,
// one score after the other: with t_0 >= t_1 >= .. a score v makes t_j the median of t_{j-1}, t_j and v; only
// a larger v goes before, so equal scores stay in order.  Then each round takes the largest of the lanes'
// first ones, of equal ones the first lane's, and that lane moves its list up.  (All rounds over all scores
// took twice the instructions, which are what bounds the kernel: 1,187,403 x 4 of 64 in fp32 175 us.)
// ALONE: one block has all rows, and places the pairs too.
template <typename T, int L, int K, bool ALONE>
__global__ __launch_bounds__(256) void k_route_top(const T *__restrict__ logits, int64_t ld, int64_t n, int experts, int k,
                                                   int normalize, int rows_per_block, int bits, int32_t *chosen,
                                                   float *gates, uint32_t *counts, int32_t *offsets, int32_t *rows, int32_t *slots)
{
    constexpr int V = VEC<T>, RPB = 256 / L, CH = 16 / V, MOST = K < 16 ? K : 16;
    __shared__ uint32_t hist[SUBMCONV_ROUTE_MAX_EXPERTS + 1];
    __shared__ uint32_t at[ALONE ? 4 : 1][SUBMCONV_ROUTE_MAX_EXPERTS + 1];
    __shared__ uint32_t lds[4];
    __shared__ int32_t numbers[RPB * K];
    __shared__ uint32_t keys[RPB * K];
    for (int i = threadIdx.x; i <= experts; i += 256) hist[i] = 0;
    __syncthreads();
    const int lane = threadIdx.x % L, g = threadIdx.x / L;
    const uint64_t group = (L == 64 ? ~0ull : (1ull << L) - 1) << (lane_id() / L * L);  // of the wave's lanes
    const int64_t first = (int64_t)blockIdx.x * rows_per_block;
    const int64_t end = first + rows_per_block < n ? first + rows_per_block : n;
    int nv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int e = lane * 16 + i * V;
        nv[i] = experts - e < 0 ? 0 : (experts - e < V ? experts - e : V);
    }
    Raw16 next[CH];
    const auto load = [&](int64_t row0) {
        const T *from = logits + (row0 + g < end ? row0 + g : end - 1) * ld + lane * 16;
#pragma unroll
        for (int i = 0; i < CH; ++i) next[i] = nv[i] ? load_raw(from + i * V, nv[i]) : Raw16{0, 0, 0, 0};
    };
    load(first);
    for (int64_t row0 = first; row0 < end; row0 += RPB) {
        uint32_t key[16], t[MOST];
        int32_t at_[MOST];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float v[V];
            unpack(next[i], v, logits);
#pragma unroll
            for (int j = 0; j < V; ++j) key[i * V + j] = j < nv[i] ? order_key(v[j]) : 0;
        }
        if (row0 + RPB < end) load(row0 + RPB);
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            t[j] = 0;
            at_[j] = 0;
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (i * V >= experts) break;
#pragma unroll
            for (int e = i * V; e < (i + 1) * V; ++e) {
                bool before[MOST];
#pragma unroll
                for (int j = 0; j < MOST; ++j) before[j] = key[e] > t[j];
#pragma unroll
                for (int j = MOST - 1; j >= 0; --j) {
                    if (j > e) continue;  // so many are not sorted yet
                    at_[j] = j > 0 && before[j > 0 ? j - 1 : 0] ? at_[j > 0 ? j - 1 : 0] : (before[j] ? lane * 16 + e : at_[j]);
                    const uint32_t high = j > 0 ? t[j > 0 ? j - 1 : 0] : 0xffffffffu, low = t[j] > key[e] ? t[j] : key[e];
                    t[j] = low < high ? low : high;  // (t_j <= t_{j-1})
                }
            }
        }
        float total = 0.0f;
        if (!normalize) {
            const uint32_t best = lanes_max<L>(t[0]);
            const float top = best > KEY_CLOSED ? key_value(best) : 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (key[i] > KEY_CLOSED) total += exp_of(key_value(key[i]) - top);
            total = lanes_sum<L>(total);
        }
        for (int j = 0; j < k; ++j) {
            const uint32_t best = lanes_max<L>(t[0]);
            bool mine = L == 1;
            if constexpr (L > 1) {
                const uint64_t with = __ballot(t[0] == best) & group;
                mine = lane_id() == (unsigned)__builtin_ctzll(with);
            }
            if (mine) {
                numbers[g * k + j] = best > KEY_CLOSED ? at_[0] : -1;
                keys[g * k + j] = best;
#pragma unroll
                for (int i = 0; i + 1 < MOST; ++i) {
                    t[i] = t[i + 1];
                    at_[i] = at_[i + 1];
                }
                t[MOST - 1] = 0;
            }
        }
        // The pairs of a wave's rows lie next to each other; no other wave sees its part of the LDS.
        wave_sync();
        if (normalize) {
            const uint32_t best = keys[g * k];
            const float top = best > KEY_CLOSED ? key_value(best) : 0.0f;
            for (int j = lane; j < k; j += L)
                if (keys[g * k + j] > KEY_CLOSED) total += exp_of(key_value(keys[g * k + j]) - top);
            total = lanes_sum<L>(total);
        }
        float gate[(K + L - 1) / L];
#pragma unroll
        for (int i = 0; i < (K + L - 1) / L; ++i) {
            const int j = i * L + lane;
            gate[i] = 0.0f;
            if (j < k) {
                const uint32_t own = keys[g * k + j], best = keys[g * k];
                if (own > KEY_CLOSED) gate[i] = exp_of(key_value(own) - key_value(best)) / total;
            }
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < (K + L - 1) / L; ++i)
            if (i * L + lane < k) keys[g * k + i * L + lane] = __float_as_uint(gate[i]);
        wave_sync();
        const int64_t w0 = row0 + (int64_t)(threadIdx.x >> 6) * (64 / L);
        const int64_t here = end - w0 < 64 / L ? end - w0 : 64 / L;
        const int base = (int)(threadIdx.x >> 6) * (64 / L) * k;
        for (int i = (int)lane_id(); i < (int)here * k; i += 64) {
            const int32_t number = numbers[base + i];
            chosen[w0 * k + i] = number;
            gates[w0 * k + i] = __uint_as_float(keys[base + i]);
            atomicAdd(&hist[number < 0 ? experts : number], 1u);
        }
        wave_sync();
    }
    __syncthreads();
    if constexpr (ALONE) {
        place_pairs(chosen, 0, n * k, k, experts, bits, at, lds, [](int) { return 0u; }, [&](int i) { return hist[i]; }, offsets, rows, slots);
    } else {
        for (int i = threadIdx.x; i <= experts; i += 256) counts[(int64_t)i * gridDim.x + blockIdx.x] = hist[i];
    }
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

// The places of each block's pairs.  SCANNED: counts are sums over the blocks already; else each block
// adds up the few that there are.
template <bool SCANNED>
__global__ __launch_bounds__(256) void k_route_place(const int32_t *__restrict__ chosen, int64_t pairs, int k, int experts, int bits,
                                                     int pairs_per_block, const uint32_t *__restrict__ counts,
                                                     const uint32_t *__restrict__ totals, int32_t *__restrict__ offsets,
                                                     int32_t *__restrict__ rows, int32_t *__restrict__ slots)
{
    __shared__ uint32_t at[4][SUBMCONV_ROUTE_MAX_EXPERTS + 1];
    __shared__ uint32_t lds[4];
    const int64_t first = (int64_t)blockIdx.x * pairs_per_block;
    const int64_t end = first + pairs_per_block < pairs ? first + pairs_per_block : pairs;
    const auto sum = [&](int bin, int blocks) {
        uint32_t s = 0;
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) s += counts[(int64_t)bin * gridDim.x + b];
        return s;
    };
    place_pairs(chosen, first, end, k, experts, bits, at, lds,
                [&](int bin) { return SCANNED ? counts[(int64_t)bin * gridDim.x + blockIdx.x] : sum(bin, blockIdx.x); },
                [&](int bin) { return SCANNED ? totals[bin] : sum(bin, gridDim.x); }, offsets, rows, slots);
}

// dL/dscore of expert e: with d_j = dgate_j gate_j,  [e = expert j] d_j - p_e sum(d)  where p is the
// softmax over the chosen experts or over all.  K: most experts of a row; their numbers, gates and
// gradients are all loaded at once.  A pair of no expert has a gate of 0, and its gradient may be anything (that of a
// logarithm of the gate is infinite): its d is 0, not 0 times that.
template <typename T, int L, int CH, int K>
__global__ __launch_bounds__(256) void k_route_bwd(const float *__restrict__ grad, const T *__restrict__ logits, int64_t ld, int64_t n,
                                                   int experts, int k, int normalize, const int32_t *__restrict__ chosen,
                                                   const float *__restrict__ gates, T *__restrict__ out, int64_t out_ld)
{
    constexpr int V = VEC<T>, RPB = 256 / L;
    const int lane = threadIdx.x % L, g = threadIdx.x / L;
    int nv[CH], e0[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int e = (i * L + lane) * V;
        nv[i] = experts - e < 0 ? 0 : (experts - e < V ? experts - e : V);
        e0[i] = nv[i] ? e : 0;
    }
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < n; row0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = row0 + g < n ? row0 + g : n - 1;
        const bool on = row0 + g < n;
        float v[CH][V], d[K], gate[K];
        int32_t number[K];
        Raw16 raw[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) raw[i] = normalize ? Raw16{0, 0, 0, 0} : load_raw(logits + row * ld + e0[i], nv[i]);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const bool there = j < k;
            const int64_t at = row * k + (there ? j : 0);
            number[j] = there ? chosen[at] : -1;
            gate[j] = gates[at];
            d[j] = grad[at];
        }
#pragma unroll
        for (int j = 0; j < K; ++j)
            if ((uint32_t)number[j] >= (uint32_t)experts && gate[j] == 0.0f) d[j] = 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (j < k) sum += d[j] * gate[j];
#pragma unroll
        for (int i = 0; i < CH; ++i) unpack(raw[i], v[i], out);
        if (!normalize) {
            float total = 0.0f;
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const uint32_t key = q < nv[i] ? order_key(v[i][q]) : 0;
                    best = best > key ? best : key;
                }
            best = lanes_max<L>(best);
            const bool open = best > KEY_CLOSED;
            const float from = open ? key_value(best) : 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    v[i][q] = q < nv[i] ? expf(v[i][q] - from) : 0.0f;
                    total += v[i][q];
                }
            total = lanes_sum<L>(total);
            const float f = open ? -sum / total : 0.0f;  // a row that is closed altogether has no gradient
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) v[i][q] *= f;
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (j >= k) break;
            const float t = gate[j] * (normalize ? d[j] - sum : d[j]);
            const int at = number[j] - lane * V;  // in the lane's first piece
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    if (at == i * L * V + q) v[i][q] += t;
        }
        if (on) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (nv[i]) store_raw(out + row * out_ld + e0[i], repack(v[i], out), nv[i]);
        }
    }
}

// Lanes a row takes in the backward pass, a power of two: eight scores a lane (two pieces in fp32).
template <typename T> constexpr int ROUTE_CH = sizeof(T) == 4 ? 2 : 1;
static int route_lanes(int experts)
{
    int lanes = 1;
    while (lanes * 8 < experts) lanes *= 2;
    return lanes;
}
#define ROUTE_LANES(GO, T)          \
    switch (lanes) {                \
    case 1: GO(T, 1); break;        \
    case 2: GO(T, 2); break;        \
    case 4: GO(T, 4); break;        \
    case 8: GO(T, 8); break;        \
    case 16: GO(T, 16); break;      \
    case 32: GO(T, 32); break;      \
    default: GO(T, 64);             \
    }
#define ROUTE_TYPES(GO) if (dtype == SUBMCONV_F32) { ROUTE_LANES(GO, float) } else { ROUTE_LANES(GO, uint16_t) }

static int route_rows(int k) { return ROUTE_PAIRS / k; }
static int64_t route_blocks(int64_t n, int k) { return (n + route_rows(k) - 1) / route_rows(k); }

size_t route_workspace(int64_t n, int experts, int k)
{
    const int64_t blocks = route_blocks(n, k);
    return blocks > 1 ? (size_t)(blocks + 1) * (experts + 1) * sizeof(uint32_t) : 0;
}

int route(const void *logits, int64_t ld, int64_t n, int experts, int k, int dtype, int normalize, int32_t *chosen, float *gates,
          int32_t *offsets, int32_t *rows, int32_t *slots, void *workspace, hipStream_t st)
{
    const int bits = bits_for(experts + 1), per_block = route_rows(k);
    int top_lanes = 1;
    while (top_lanes * 16 < experts) top_lanes *= 2;
    const int64_t blocks = route_blocks(n, k);
    uint32_t *counts = (uint32_t *)workspace, *totals = counts + blocks * (experts + 1);
#define TOP(T, L, K, ALONE)                                                                                                \
    hipLaunchKernelGGL((k_route_top<T, L, K, ALONE>), dim3((unsigned)blocks), dim3(256), 0, st, (const T *)logits, ld, n, experts, k, \
                       normalize, per_block, bits, chosen, gates, counts, offsets, rows, slots)
#define ALL(T, L, K) if (blocks == 1) TOP(T, L, K, true); else TOP(T, L, K, false)
#define GO(T, L) if (k <= 2) { ALL(T, L, 2); } else if (k <= 4) { ALL(T, L, 4); } else if (k <= 8) { ALL(T, L, 8); } else { ALL(T, L, 16); }
    switch (top_lanes) {
    case 1: if (dtype == SUBMCONV_F32) { GO(float, 1) } else { GO(uint16_t, 1) } break;
    case 2: if (dtype == SUBMCONV_F32) { GO(float, 2) } else { GO(uint16_t, 2) } break;
    case 4: if (dtype == SUBMCONV_F32) { GO(float, 4) } else { GO(uint16_t, 4) } break;
    case 8: if (dtype == SUBMCONV_F32) { GO(float, 8) } else { GO(uint16_t, 8) } break;
    case 16: if (dtype == SUBMCONV_F32) { GO(float, 16) } else { GO(uint16_t, 16) } break;
    default: if (dtype == SUBMCONV_F32) { GO(float, 32) } else { GO(uint16_t, 32) }
    }
#undef GO
#undef ALL
#undef TOP
    SC_LAUNCHED("route");
    if (blocks == 1) return SUBMCONV_OK;
    const bool scan = blocks > 64;
    if (scan) {
        hipLaunchKernelGGL(k_route_scan, dim3(experts + 1), dim3(256), 0, st, counts, (int)blocks, totals);
        SC_LAUNCHED("route sums");
    }
    const dim3 grid((unsigned)blocks);
    if (scan) hipLaunchKernelGGL(k_route_place<true>, grid, dim3(256), 0, st, chosen, n * k, k, experts, bits, per_block * k, counts, totals, offsets, rows, slots);
    else hipLaunchKernelGGL(k_route_place<false>, grid, dim3(256), 0, st, chosen, n * k, k, experts, bits, per_block * k, counts, totals, offsets, rows, slots);
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
    const int lanes = route_lanes(experts);
    const int64_t rpb = 256 / lanes, blocks = (n + rpb - 1) / rpb;
    const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
#define BACK(T, L, K)                                                                                                          \
    hipLaunchKernelGGL((k_route_bwd<T, L, ROUTE_CH<T>, K>), grid, dim3(256), 0, st, grad, (const T *)logits, ld, n, experts, k, normalize, chosen, \
                       gates, (T *)out, out_ld)
#define GO(T, L) if (k <= 2) BACK(T, L, 2); else if (k <= 4) BACK(T, L, 4); else if (k <= 8) BACK(T, L, 8); else BACK(T, L, 16)
    ROUTE_TYPES(GO)
#undef GO
#undef BACK
    SC_LAUNCHED("route_backward");
    return SUBMCONV_OK;
}

}  // namespace sc
