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
// some 60 instructions, about what a piece may take at the memory's rate).  Two rows a lane at a time keep enough loads
// in flight; the launch is as many blocks as the card holds at once of the bf16 kernels for paired halves, which have the
// most registers, so that none waits for a place (of the others it would hold up to twice as many; not tried).
//
// Measured: forward 20,384 x 16 heads of 128 in bf16, packed, 34 us (4.9 TB/s, the rate of a copy); 400,311 x 12 of 64,
// paired halves, bf16: forward 248 us (5.0 TB/s), backward 419 (4.4; one row a lane 462, twice the blocks 445 to 460), dw's
// sums 5; fp32 447 (5.5) and 689 (5.4); neighbours as pairs, bf16 295 (4.2) and 481 (3.8), fp32 494 (5.0) and 854 (4.3).
// 450 x 4 of 64 in fp32: 4 us, a launch and three memory latencies.
#include "headnorm.h"

namespace sc {

// Which row of the weight a head takes.
__device__ __forceinline__ int weight_row(const HeadNormArgs &A, int h)
{
    return A.q_heads ? h >= A.q_heads : (A.weight_rows > 1 ? h : 0);
}

// The angles of a block's rows in LDS, [rows][used], two sets in turn.  A thread forms its share of the next
// rows' angles while the present rows are worked on; the position of its first one is loaded a turn earlier
// still, so that no wave waits for it.
struct Angles {
    float2 *tab;
    int used, many;     // pairs that turn, angles of a set
    int r, p, axis;     // the thread's first angle: row and pair
    float freq;
    int32_t position;

    __device__ __forceinline__ Angles(const HeadNormArgs &A, float2 *lds, int rows) : tab(lds)
    {
        used = A.ax.end[SUBMCONV_ROTARY_MAX_AXES - 1];
        many = rows * used;
        r = used ? threadIdx.x / used : 0;
        p = threadIdx.x - r * used;
        axis = rotary_axis(A.ax, p);
        freq = (int)threadIdx.x < many ? A.freqs[p] : 0.0f;
        position = 0;
    }
    // The first position of the rows from row0 on.
    __device__ __forceinline__ void load(const HeadNormArgs &A, int64_t row0)
    {
        if ((int)threadIdx.x < many) position = A.pos[(row0 + r < A.n ? row0 + r : A.n - 1) * A.pos_row + axis];
    }
    // The angles of the rows from row0 on, into set k.
    __device__ __forceinline__ void form(const HeadNormArgs &A, int64_t row0, int k)
    {
        if ((int)threadIdx.x < many) {
            float c, s;
            turn(position, freq, false, &c, &s);
            tab[k * many + threadIdx.x] = make_float2(c, s);
        }
        for (int i = threadIdx.x + 256; i < many; i += 256) {
            const int row = i / used, q = i - row * used;
            float c, s;
            turn(A.pos[(row0 + row < A.n ? row0 + row : A.n - 1) * A.pos_row + rotary_axis(A.ax, q)], A.freqs[q], false, &c, &s);
            tab[k * many + i] = make_float2(c, s);
        }
    }
};

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

// Squares leave fp32 above 2^64 and lose bits below 2^-63, though 1 / sqrt of their mean is an ordinary number there.  A mean
// of 2^-100 to 2^120 is right (512 squares at most, and those below 2^-126 do not count).
__device__ __forceinline__ bool head_mean_fits(float mean) { return mean >= 0x1p-100f && mean <= 0x1p+120f; }

// 1 / sqrt(mean + eps) of a head whose mean is not: of the squares of c times the head, c a power of two.  2^-70 takes the
// largest values to 2^58, whose squares' sum stays below 2^126; 2^90 takes those of a mean below 2^-100 to 2^45 at most.
template <int L, int P, int V>
__device__ __forceinline__ float head_rstd_far(const float (&v)[P][V], float mean, float dim, float eps)
{
    const float c = mean > 1.0f ? 0x1p-70f : 0x1p+90f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float t = v[i][j] * c;
            s += t * t;
        }
    return rsqrtf(lanes_sum<L>(s) / dim + eps * c * c) * c;
}

constexpr int HEAD_ROWS = 2;  // rows of a lane at a time, their loads issued together

// out may be x (so neither is restrict).
template <typename T, int L, int P, bool SPLIT>
__global__ __launch_bounds__(256) void k_head_norm(HeadNormArgs A)
{
    constexpr int V = VEC<T>, U = HEAD_ROWS;
    extern __shared__ __attribute__((aligned(16))) float2 tab[];
    const HeadPieces<T, L, P, SPLIT> at(A.dim);
    const int group = threadIdx.x / L, r = group / A.hb, h = blockIdx.y * A.hb + group - r * A.hb;
    const bool here = r < A.rb && h < A.heads;
    const int hh = here ? h : 0;
    Angles angles(A, tab, U * A.rb);
    const int used = angles.used;
    const T *x = (const T *)A.x + hh * A.x_head;
    T *out = (T *)A.out + hh * A.out_head;
    const int64_t step = (int64_t)gridDim.x * A.rb * U;
    int64_t row0 = (int64_t)blockIdx.x * A.rb * U;
    const auto row_at = [&](int64_t first, int u) { const int64_t row = first + u * A.rb + r; return row < A.n ? row : A.n - 1; };
    Raw16 next[U][P];
    const auto load = [&](int64_t first) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < P; ++i) next[u][i] = load_raw(x + row_at(first, u) * A.x_row + at.e[i], at.nv[i]);
    };
    angles.load(A, row0);
    load(row0);
    float w[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) w[i][j] = A.w && j < at.nv[i] ? param(A.w, A.pdtype, weight_row(A, hh) * A.dim + at.e[i] + j) : 1.0f;
    if (used) {
        angles.form(A, row0, 0);
        angles.load(A, row0 + step);
    }
    const float dim = (float)A.dim;
    for (int k = 0; row0 < A.n; row0 += step, k ^= 1) {
        float v[U][P][V], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                unpack(next[u][i], v[u][i], x);
#pragma unroll
                for (int j = 0; j < V; ++j) s[u] += v[u][i][j] * v[u][i][j];  // zero past the head's end
            }
        }
        if (used) __syncthreads();  // set k is written; the other is read no more
        if (row0 + step < A.n) {
            load(row0 + step);
            if (used) {
                angles.form(A, row0 + step, k ^ 1);
                angles.load(A, row0 + 2 * step);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float mean = lanes_sum<L>(s[u]) / dim + A.eps;
            float rs = rsqrtf(mean);
            // (a wave's branch, for few instructions: 20,384 x 16 heads of 128, packed, 31.2 -> 31.5 us; always both ways 33.8)
            if (__builtin_expect(__ballot(!head_mean_fits(mean)) != 0, 0)) {
                const float far = head_rstd_far<L>(v[u], mean, dim, A.eps);
                rs = head_mean_fits(mean) ? rs : far;
            }
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) v[u][i][j] = v[u][i][j] * rs * w[i][j];
            at.turn_pairs(v[u], tab + k * angles.many + (u * A.rb + (r < A.rb ? r : 0)) * used, used, 1.0f);
            const int64_t row = row0 + u * A.rb + r;
            if (here && row < A.n) {
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if (at.nv[i]) store_raw(out + row * A.out_row + at.e[i], repack(v[u][i], x), at.nv[i]);
                if (A.rstd && at.lane == 0) A.rstd[row * A.heads + h] = rs;
            }
        }
    }
}

// dx, and the block's share of dw over its rows: summed in registers, then over the block's lanes
// of one weight in a fixed order through LDS, and over blocks by k_head_wgrad.  No atomics.
// out may be g.
template <typename T, int L, int P, bool SPLIT>
__global__ __launch_bounds__(256) void k_head_norm_bwd(HeadNormArgs A)
{
    constexpr int V = VEC<T>, U = HEAD_ROWS;
    extern __shared__ __attribute__((aligned(16))) float2 tab[];
    const HeadPieces<T, L, P, SPLIT> at(A.dim);
    const int group = threadIdx.x / L, r = group / A.hb, h = blockIdx.y * A.hb + group - r * A.hb;
    const bool here = r < A.rb && h < A.heads;
    const int hh = here ? h : 0;
    Angles angles(A, tab, U * A.rb);
    const int used = angles.used;
    const T *x = (const T *)A.x + hh * A.x_head, *g = (const T *)A.g + hh * A.g_head;
    T *out = (T *)A.out + hh * A.out_head;
    const int64_t step = (int64_t)gridDim.x * A.rb * U;
    int64_t row0 = (int64_t)blockIdx.x * A.rb * U;
    const auto row_at = [&](int64_t first, int u) { const int64_t row = first + u * A.rb + r; return row < A.n ? row : A.n - 1; };
    Raw16 nx[U][P], ng[U][P];
    float nr[U];
    const auto load = [&](int64_t first) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row_at(first, u);
            nr[u] = A.rstd[row * A.heads + hh];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                nx[u][i] = load_raw(x + row * A.x_row + at.e[i], at.nv[i]);
                ng[u][i] = load_raw(g + row * A.g_row + at.e[i], at.nv[i]);
            }
        }
    };
    angles.load(A, row0);
    load(row0);
    float w[P][V], dw[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[i][j] = A.w && j < at.nv[i] ? param(A.w, A.pdtype, weight_row(A, hh) * A.dim + at.e[i] + j) : 1.0f;
            dw[i][j] = 0.0f;
        }
    if (used) {
        angles.form(A, row0, 0);
        angles.load(A, row0 + step);
    }
    const float dim = (float)A.dim;
    for (int k = 0; row0 < A.n; row0 += step, k ^= 1) {
        float hat[U][P][V], g_[U][P][V], rs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rs[u] = nr[u];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                unpack(nx[u][i], hat[u][i], x);
                unpack(ng[u][i], g_[u][i], x);
            }
        }
        if (used) __syncthreads();  // set k is written; the other is read no more
        if (row0 + step < A.n) {
            load(row0 + step);
            if (used) {
                angles.form(A, row0 + step, k ^ 1);
                angles.load(A, row0 + 2 * step);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * A.rb + r;
            const bool on = here && row < A.n;
            at.turn_pairs(g_[u], tab + k * angles.many + (u * A.rb + (r < A.rb ? r : 0)) * used, used, -1.0f);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    hat[u][i][j] *= rs[u];
                    if (on) dw[i][j] += g_[u][i][j] * hat[u][i][j];
                    g_[u][i][j] *= w[i][j];
                    s += g_[u][i][j] * hat[u][i][j];
                }
            s = lanes_sum<L>(s) / dim;
            if (on) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
#pragma unroll
                    for (int j = 0; j < V; ++j) g_[u][i][j] = rs[u] * (g_[u][i][j] - hat[u][i][j] * s);
                    if (at.nv[i]) store_raw(out + row * A.out_row + at.e[i], repack(g_[u][i], x), at.nv[i]);
                }
            }
        }
    }
    if (!A.partial) return;
    // [group][dim] in LDS, in the angles' place
    constexpr int PAD = L * P * V;
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
static HeadShape head_shape(int heads, int dim, int dtype, int split)
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
    return s;
}

constexpr int64_t HEAD_FWD_BLOCKS = 1024, HEAD_BWD_BLOCKS = 512;
static int64_t head_blocks(int64_t n, const HeadShape &s, int64_t most)
{
    const int64_t rows = s.rb * HEAD_ROWS, b = (n + rows - 1) / rows, m = most / s.chunks > 0 ? most / s.chunks : 1;
    return b < m ? b : m;
}

// Rows of partial sums the backward pass leaves.
static int64_t head_partials(int64_t n, const HeadShape &s, int heads, int weight_rows, int q_heads)
{
    return head_blocks(n, s, HEAD_BWD_BLOCKS) * (weight_rows == heads && !q_heads ? 1 : s.chunks);
}

size_t head_norm_bwd_workspace(int64_t n, int heads, int dim, int dtype, int weight_rows, int q_heads)
{
    int64_t most = 0;  // of both orders of pairs
    for (int split = 0; split < 2; ++split) {
        const int64_t p = head_partials(n, head_shape(heads, dim, dtype, split), heads, weight_rows, q_heads);
        most = p > most ? p : most;
    }
    return (size_t)most * weight_rows * dim * sizeof(float);
}

// Bytes of LDS: two sets of angles, at most 64 KB (256 / L rows a block of at most L V pairs each, HEAD_ROWS of them a lane).
static size_t head_lds(const HeadNormArgs &A, const HeadShape &s) { return (size_t)2 * HEAD_ROWS * s.rb * A.ax.end[SUBMCONV_ROTARY_MAX_AXES - 1] * sizeof(float2); }

#define HEAD_LANES(K, T, P, SPLIT)                                                                  \
    switch (s.lanes) {                                                                              \
    case 2: hipLaunchKernelGGL((K<T, 2, P, SPLIT>), grid, dim3(256), lds, st, A); break;              \
    case 4: hipLaunchKernelGGL((K<T, 4, P, SPLIT>), grid, dim3(256), lds, st, A); break;              \
    case 8: hipLaunchKernelGGL((K<T, 8, P, SPLIT>), grid, dim3(256), lds, st, A); break;              \
    case 16: hipLaunchKernelGGL((K<T, 16, P, SPLIT>), grid, dim3(256), lds, st, A); break;            \
    case 32: hipLaunchKernelGGL((K<T, 32, P, SPLIT>), grid, dim3(256), lds, st, A); break;            \
    default: hipLaunchKernelGGL((K<T, 64, P, SPLIT>), grid, dim3(256), lds, st, A);                   \
    }
#define HEAD_KERNELS(K)                                                                             \
    if (dtype == SUBMCONV_F32) {                                                                    \
        if (split) { HEAD_LANES(K, float, 2, true) }                                                \
        else if (s.pieces == 2) hipLaunchKernelGGL((K<float, 64, 2, false>), grid, dim3(256), lds, st, A); \
        else { HEAD_LANES(K, float, 1, false) }                                                     \
    } else {                                                                                        \
        if (split) { HEAD_LANES(K, uint16_t, 2, true) }                                             \
        else { HEAD_LANES(K, uint16_t, 1, false) }                                                  \
    }

int head_norm(HeadNormArgs A, int dtype, int split, hipStream_t st)
{
    const HeadShape s = head_shape(A.heads, A.dim, dtype, split);
    A.hb = s.hb;
    A.rb = s.rb;
    const dim3 grid((unsigned)head_blocks(A.n, s, HEAD_FWD_BLOCKS), (unsigned)s.chunks);
    const size_t lds = head_lds(A, s);
    HEAD_KERNELS(k_head_norm)
    SC_LAUNCHED("head_norm_rotary");
    return SUBMCONV_OK;
}

int head_norm_backward(HeadNormArgs A, int dtype, int split, void *dw, hipStream_t st)
{
    const HeadShape s = head_shape(A.heads, A.dim, dtype, split);
    A.hb = s.hb;
    A.rb = s.rb;
    if (!dw) A.partial = nullptr;
    if (A.n > 0) {
        const dim3 grid((unsigned)head_blocks(A.n, s, HEAD_BWD_BLOCKS), (unsigned)s.chunks);
        const size_t sums = dw ? (size_t)256 * s.pieces * (dtype == SUBMCONV_F32 ? 4 : 8) * sizeof(float) : 0, angles = head_lds(A, s);
        const size_t lds = sums > angles ? sums : angles;
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
