// The root-mean-square norm of each head of a row, with the rotation by the row's positions in
// the same pass, and its backward pass.  For a head x of `dim` elements and its weight w:
//
//   r = 1 / sqrt(sum x^2 / dim + eps),  h = x r,  y = R(h w)        (R: the rotation of rotary.hip)
//   u = R^-1 g,  dw = sum over rows (and heads of one weight) u h,
//   dx = r (u w - h sum(u w h) / dim)
//
// Both passes are bound by memory: x is read once and y written once; backward reads x and g and
// writes dx.  L lanes hold a head in registers, 16 bytes a piece, in fp32.  A block's lanes are HB
// heads of RB rows; a lane keeps its head and walks rows, so that the weight and the sums of dw
// stay in registers.  The heads of a row turn by the same angles: the block forms the sines and
// cosines of its RB rows once, in LDS, while the rows before them are worked on (an angle costs
// some 60 instructions, about what a piece may take at the memory's rate).
#include "headnorm.h"

namespace sc {

// Which row of the weight a head takes.
__device__ __forceinline__ int weight_row(const HeadNormArgs &A, int h)
{
    return A.q_heads ? h >= A.q_heads : (A.weight_rows > 1 ? h : 0);
}

// cos and sin of the pairs of RB rows from row0 on, into tab [rb][used].
__device__ __forceinline__ void form_angles(const HeadNormArgs &A, int64_t row0, float2 *tab)
{
    const int used = A.ax.end[SUBMCONV_ROTARY_MAX_AXES - 1];
    for (int i = threadIdx.x; i < A.rb * used; i += 256) {
        const int r = i / used, p = i - r * used;
        const int64_t row = row0 + r < A.n ? row0 + r : A.n - 1;
        float c, s;
        turn(A.pos[row * A.pos_row + rotary_axis(A.ax, p)], A.freqs[p], false, &c, &s);
        tab[i] = make_float2(c, s);
    }
}

// A lane's elements of a head: P pieces of V.  SPLIT: the same piece of both halves (a pair is
// elements j of both), otherwise pieces L apart (a pair is two neighbours).
template <typename T, int L, int P, bool SPLIT>
struct HeadPieces {
    static constexpr int V = VEC<T>;
    int e[P], nv[P], lane;

    __device__ __forceinline__ explicit HeadPieces(int dim)
    {
        lane = threadIdx.x % L;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int at = SPLIT ? lane * V : (i * L + lane) * V, end = SPLIT ? dim / 2 : dim;
            nv[i] = end - at < 0 ? 0 : (end - at < V ? end - at : V);
            e[i] = (SPLIT && i ? dim / 2 : 0) + (nv[i] ? at : 0);
        }
    }
    // Turn the pairs of v by the angles of tab [used], forwards (sign 1) or back (-1).
    __device__ __forceinline__ void turn_pairs(float (&v)[P][V], const float2 *tab, int used, float sign) const
    {
        if constexpr (SPLIT) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int p = lane * V + j;
                if (p >= used) continue;
                const float2 t = tab[p];
                const float a = v[0][j], b = v[P - 1][j], s = t.y * sign;
                v[0][j] = a * t.x - b * s;
                v[P - 1][j] = a * s + b * t.x;
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const int p = (i * L + lane) * (V / 2) + j;
                    if (p >= used) continue;
                    const float2 t = tab[p];
                    const float a = v[i][2 * j], b = v[i][2 * j + 1], s = t.y * sign;
                    v[i][2 * j] = a * t.x - b * s;
                    v[i][2 * j + 1] = a * s + b * t.x;
                }
        }
    }
};

constexpr int HEAD_TAB = 2048;  // angles of a block's rows that fit in LDS, twice

// out may be x (so neither is restrict).
template <typename T, int L, int P, bool SPLIT>
__global__ __launch_bounds__(256) void k_head_norm(HeadNormArgs A)
{
    constexpr int V = VEC<T>;
    __shared__ float2 tab[2][HEAD_TAB];
    const HeadPieces<T, L, P, SPLIT> at(A.dim);
    const int used = A.ax.end[SUBMCONV_ROTARY_MAX_AXES - 1];
    const int group = threadIdx.x / L, r = group / A.hb, h = blockIdx.y * A.hb + group - r * A.hb;
    const bool here = r < A.rb && h < A.heads;
    const int hh = here ? h : 0;
    float w[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) w[i][j] = A.w && j < at.nv[i] ? param(A.w, A.pdtype, weight_row(A, hh) * A.dim + at.e[i] + j) : 1.0f;
    const T *x = (const T *)A.x + hh * A.x_head;
    T *out = (T *)A.out + hh * A.out_head;
    const int64_t step = (int64_t)gridDim.x * A.rb;
    int64_t row0 = (int64_t)blockIdx.x * A.rb;
    const auto row_at = [&](int64_t first) { return first + r < A.n ? first + r : A.n - 1; };
    Raw16 next[P];
#pragma unroll
    for (int i = 0; i < P; ++i) next[i] = load_raw(x + row_at(row0) * A.x_row + at.e[i], at.nv[i]);
    if (used) form_angles(A, row0, tab[0]);
    const float dim = (float)A.dim;
    for (int k = 0; row0 < A.n; row0 += step, k ^= 1) {
        float v[P][V], s = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            unpack(next[i], v[i], x);
#pragma unroll
            for (int j = 0; j < V; ++j) s += v[i][j] * v[i][j];  // zero past the head's end
        }
        if (used) __syncthreads();  // tab[k] is written; tab[k ^ 1] is read no more
        if (row0 + step < A.n) {
#pragma unroll
            for (int i = 0; i < P; ++i) next[i] = load_raw(x + row_at(row0 + step) * A.x_row + at.e[i], at.nv[i]);
            if (used) form_angles(A, row0 + step, tab[k ^ 1]);
        }
        const float rs = rsqrtf(lanes_sum<L>(s) / dim + A.eps);
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * rs * w[i][j];
        at.turn_pairs(v, tab[k] + (r < A.rb ? r : 0) * used, used, 1.0f);
        const int64_t row = row0 + r;
        if (here && row < A.n) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (at.nv[i]) store_raw(out + row * A.out_row + at.e[i], repack(v[i], x), at.nv[i]);
            if (A.rstd && at.lane == 0) A.rstd[row * A.heads + h] = rs;
        }
    }
}

// dx, and the block's share of dw over its rows: summed in registers, then over the block's lanes
// of one weight in a fixed order through LDS, and over blocks by k_head_wgrad.  No atomics.
// out may be g.
template <typename T, int L, int P, bool SPLIT>
__global__ __launch_bounds__(256) void k_head_norm_bwd(HeadNormArgs A)
{
    constexpr int V = VEC<T>;
    __shared__ float2 tab[2][HEAD_TAB];
    const HeadPieces<T, L, P, SPLIT> at(A.dim);
    const int used = A.ax.end[SUBMCONV_ROTARY_MAX_AXES - 1];
    const int group = threadIdx.x / L, r = group / A.hb, h = blockIdx.y * A.hb + group - r * A.hb;
    const bool here = r < A.rb && h < A.heads;
    const int hh = here ? h : 0;
    float w[P][V], dw[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[i][j] = A.w && j < at.nv[i] ? param(A.w, A.pdtype, weight_row(A, hh) * A.dim + at.e[i] + j) : 1.0f;
            dw[i][j] = 0.0f;
        }
    const T *x = (const T *)A.x + hh * A.x_head, *g = (const T *)A.g + hh * A.g_head;
    T *out = (T *)A.out + hh * A.out_head;
    const int64_t step = (int64_t)gridDim.x * A.rb;
    int64_t row0 = (int64_t)blockIdx.x * A.rb;
    const auto row_at = [&](int64_t first) { return first + r < A.n ? first + r : A.n - 1; };
    Raw16 nx[P], ng[P];
    float nr = A.rstd[row_at(row0) * A.heads + hh];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        nx[i] = load_raw(x + row_at(row0) * A.x_row + at.e[i], at.nv[i]);
        ng[i] = load_raw(g + row_at(row0) * A.g_row + at.e[i], at.nv[i]);
    }
    if (used) form_angles(A, row0, tab[0]);
    const float dim = (float)A.dim;
    for (int k = 0; row0 < A.n; row0 += step, k ^= 1) {
        const int64_t row = row0 + r;
        const bool on = here && row < A.n;
        float hat[P][V], u[P][V];
        const float rs = nr;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            unpack(nx[i], hat[i], x);
            unpack(ng[i], u[i], x);
        }
        if (used) __syncthreads();  // tab[k] is written; tab[k ^ 1] is read no more
        if (row0 + step < A.n) {
            nr = A.rstd[row_at(row0 + step) * A.heads + hh];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                nx[i] = load_raw(x + row_at(row0 + step) * A.x_row + at.e[i], at.nv[i]);
                ng[i] = load_raw(g + row_at(row0 + step) * A.g_row + at.e[i], at.nv[i]);
            }
            if (used) form_angles(A, row0 + step, tab[k ^ 1]);
        }
        at.turn_pairs(u, tab[k] + (r < A.rb ? r : 0) * used, used, -1.0f);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                hat[i][j] *= rs;
                if (on) dw[i][j] += u[i][j] * hat[i][j];
                u[i][j] *= w[i][j];
                s += u[i][j] * hat[i][j];
            }
        s = lanes_sum<L>(s) / dim;
        if (on) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
#pragma unroll
                for (int j = 0; j < V; ++j) u[i][j] = rs * (u[i][j] - hat[i][j] * s);
                if (at.nv[i]) store_raw(out + row * A.out_row + at.e[i], repack(u[i], x), at.nv[i]);
            }
        }
    }
    if (!A.partial) return;
    // [group][dim] in LDS, in the angles' place
    constexpr int GROUPS = 256 / L, PAD = L * P * V;
    static_assert(GROUPS * PAD <= 2 * HEAD_TAB * 2, "the lanes' sums fit");
    float *red = (float *)tab;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < at.nv[i]) red[group * PAD + at.e[i] + j] = dw[i][j];
    __syncthreads();
    const int h0 = blockIdx.y * A.hb, many = A.heads - h0 < A.hb ? A.heads - h0 : A.hb;
    if (A.weight_rows == A.heads && !A.q_heads) {  // each head's own
        float *mine = A.partial + (int64_t)blockIdx.x * A.weight_rows * A.dim;
        for (int i = threadIdx.x; i < many * A.dim; i += 256) {
            const int j = i / A.dim, e = i - j * A.dim;
            float s = 0.0f;
            for (int q = 0; q < A.rb; ++q) s += red[(q * A.hb + j) * PAD + e];
            mine[(h0 + j) * A.dim + e] = s;
        }
    } else {
        float *mine = A.partial + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * A.weight_rows * A.dim;
        const int first = A.q_heads ? (A.q_heads - h0 < 0 ? 0 : (A.q_heads - h0 < many ? A.q_heads - h0 : many)) : many;
        for (int i = threadIdx.x; i < A.weight_rows * A.dim; i += 256) {
            const int j = i / A.dim, e = i - j * A.dim;
            float s = 0.0f;
            for (int q = 0; q < A.rb; ++q)
                for (int m = j ? first : 0; m < (j ? many : first); ++m) s += red[(q * A.hb + m) * PAD + e];
            mine[j * A.dim + e] = s;
        }
    }
}

// Column sums of partial [blocks][cols] in a fixed order: 16 columns a block, 16 threads to a
// column.  No blocks (an empty set) leaves zeros.
__global__ __launch_bounds__(256) void k_head_wgrad(const float *__restrict__ partial, int blocks, int cols,
                                                    void *__restrict__ dw, int pdtype)
{
    __shared__ float red[16][17];
    const int col = blockIdx.x * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4;
    float s = 0.0f;
    if (col < cols) {
#pragma unroll 8
        for (int b = part; b < blocks; b += 16) s += partial[(int64_t)b * cols + col];
    }
    red[part][threadIdx.x & 15] = s;
    __syncthreads();
    if (part == 0 && col < cols) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = red[i][threadIdx.x];
#pragma unroll
        for (int o = 8; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) v[i] += v[i + o];
        set_param(dw, pdtype, col, v[0]);
    }
}

// Lanes a head takes, and how a block's lanes divide into heads and rows.
struct HeadShape {
    int lanes, pieces, hb, rb, chunks;
};
static HeadShape head_shape(int heads, int dim, int dtype, int split, int used)
{
    const int v = dtype == SUBMCONV_F32 ? 4 : 8, span = split ? dim / 2 : dim;
    HeadShape s;
    const int all = (span + v - 1) / v;
    s.lanes = 2;
    while (s.lanes < all && s.lanes < 64) s.lanes *= 2;
    s.pieces = split ? 2 : (all > 64 ? 2 : 1);
    const int groups = 256 / s.lanes;
    s.chunks = (heads + groups - 1) / groups;
    s.hb = (heads + s.chunks - 1) / s.chunks;
    s.rb = groups / s.hb;
    if (used && s.rb * used > HEAD_TAB) s.rb = HEAD_TAB / used;  // (used <= 256: eight rows at least)
    return s;
}

constexpr int64_t HEAD_FWD_BLOCKS = 2048, HEAD_BWD_BLOCKS = 1024;
static int64_t head_blocks(int64_t n, const HeadShape &s, int64_t most)
{
    const int64_t b = (n + s.rb - 1) / s.rb, m = most / s.chunks > 0 ? most / s.chunks : 1;
    return b < m ? b : m;
}

// Rows of partial sums the backward pass leaves.
static int64_t head_partials(int64_t n, const HeadShape &s, int heads, int weight_rows, int q_heads)
{
    return head_blocks(n, s, HEAD_BWD_BLOCKS) * (weight_rows == heads && !q_heads ? 1 : s.chunks);
}

size_t head_norm_bwd_workspace(int64_t n, int heads, int dim, int dtype, int weight_rows, int q_heads)
{
    // (the larger of both orders of pairs and any sections)
    int64_t most = 0;
    for (int split = 0; split < 2; ++split)
        for (int used = 0; used <= dim / 2; used += dim / 2) {
            const int64_t p = head_partials(n, head_shape(heads, dim, dtype, split, used), heads, weight_rows, q_heads);
            most = p > most ? p : most;
        }
    return (size_t)most * weight_rows * dim * sizeof(float);
}

#define HEAD_LANES(K, T, P, SPLIT)                                                                  \
    switch (s.lanes) {                                                                              \
    case 2: hipLaunchKernelGGL((K<T, 2, P, SPLIT>), grid, dim3(256), 0, st, A); break;              \
    case 4: hipLaunchKernelGGL((K<T, 4, P, SPLIT>), grid, dim3(256), 0, st, A); break;              \
    case 8: hipLaunchKernelGGL((K<T, 8, P, SPLIT>), grid, dim3(256), 0, st, A); break;              \
    case 16: hipLaunchKernelGGL((K<T, 16, P, SPLIT>), grid, dim3(256), 0, st, A); break;            \
    case 32: hipLaunchKernelGGL((K<T, 32, P, SPLIT>), grid, dim3(256), 0, st, A); break;            \
    default: hipLaunchKernelGGL((K<T, 64, P, SPLIT>), grid, dim3(256), 0, st, A);                   \
    }
#define HEAD_KERNELS(K)                                                                             \
    if (dtype == SUBMCONV_F32) {                                                                    \
        if (split) { HEAD_LANES(K, float, 2, true) }                                                \
        else if (s.pieces == 2) hipLaunchKernelGGL((K<float, 64, 2, false>), grid, dim3(256), 0, st, A); \
        else { HEAD_LANES(K, float, 1, false) }                                                     \
    } else {                                                                                        \
        if (split) { HEAD_LANES(K, uint16_t, 2, true) }                                             \
        else { HEAD_LANES(K, uint16_t, 1, false) }                                                  \
    }

int head_norm(HeadNormArgs A, int dtype, int split, hipStream_t st)
{
    const HeadShape s = head_shape(A.heads, A.dim, dtype, split, A.ax.end[SUBMCONV_ROTARY_MAX_AXES - 1]);
    A.hb = s.hb;
    A.rb = s.rb;
    const dim3 grid((unsigned)head_blocks(A.n, s, HEAD_FWD_BLOCKS), (unsigned)s.chunks);
    HEAD_KERNELS(k_head_norm)
    SC_LAUNCHED("head_norm_rotary");
    return SUBMCONV_OK;
}

int head_norm_backward(HeadNormArgs A, int dtype, int split, void *dw, hipStream_t st)
{
    const HeadShape s = head_shape(A.heads, A.dim, dtype, split, A.ax.end[SUBMCONV_ROTARY_MAX_AXES - 1]);
    A.hb = s.hb;
    A.rb = s.rb;
    if (!dw) A.partial = nullptr;
    if (A.n > 0) {
        const dim3 grid((unsigned)head_blocks(A.n, s, HEAD_BWD_BLOCKS), (unsigned)s.chunks);
        HEAD_KERNELS(k_head_norm_bwd)
        SC_LAUNCHED("head_norm_rotary_backward");
    }
    if (dw) {
        const int cols = A.weight_rows * A.dim;
        hipLaunchKernelGGL(k_head_wgrad, dim3((unsigned)((cols + 15) / 16)), dim3(256), 0, st, A.partial,
                           A.n > 0 ? (int)head_partials(A.n, s, A.heads, A.weight_rows, A.q_heads) : 0, cols, dw, A.pdtype);
        SC_LAUNCHED("head_norm_rotary_backward sums");
    }
    return SUBMCONV_OK;
}

}  // namespace sc
