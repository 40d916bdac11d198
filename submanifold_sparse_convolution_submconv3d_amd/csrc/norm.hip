// Layer normalisation of feature rows and its backward pass.
//
//   mean = sum x / C,  r = 1 / sqrt(sum (x - mean)^2 / C + eps),  h = (x - mean) r
//   y = h w + b
//   dx = r (g w - sum(g w) / C - h sum(g w h) / C),  dw = sum over rows g h,  db = sum over rows g
//
// Both passes are bound by memory: a row is read once into registers (16 bytes a lane
// at a time), its statistics are formed there in fp32 (the variance from the centred
// values, so a large common offset costs no accuracy), and the result is written once.
#include "rowvec.h"

namespace sc {

// A parameter vector's element (fp32 or bf16) as fp32.
__device__ __forceinline__ float param(const void *p, int dtype, int i)
{
    return dtype == SUBMCONV_F32 ? ((const float *)p)[i] : bf16_to_f32(((const uint16_t *)p)[i]);
}

__device__ __forceinline__ void set_param(void *p, int dtype, int i, float v)
{
    if (!p) return;
    if (dtype == SUBMCONV_F32)
        ((float *)p)[i] = v;
    else
        ((uint16_t *)p)[i] = f32_to_bf16(v);
}

// Sum of v over the TPR threads of a row.  TPR = 256: the whole block, through LDS;
// `slot` alternates between the two halves of `part`, so one barrier a sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *part, int slot)
{
    if constexpr (TPR <= 64) return lanes_sum<TPR>(v);
    v = lanes_sum<64>(v);
    float *p = part + 4 * slot;
    if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
    __syncthreads();
    return (p[0] + p[1]) + (p[2] + p[3]);
}

// TPR threads hold a row, CH pieces of 16 bytes each; a block of 256 walks rows in
// grid-sized strides with the next rows' loads issued before the current rows' sums.
// y may be x (so neither is restrict).
// 1,187,403 x 64 bf16: 56 us, 5.4 TB/s (a plain device copy reaches 4.8 to 4.9).
template <typename T, int CH, int TPR>
__global__ __launch_bounds__(256) void k_norm(const T *x, int64_t ldx, int64_t n, int c,
                                              const void *__restrict__ w, const void *__restrict__ b, int pdtype,
                                              float eps, T *y, int64_t ldy, float2 *__restrict__ stats)
{
    constexpr int V = VEC<T>, RPB = 256 / TPR;
    __shared__ float part[8];
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    int nv[CH];
    float wr[CH][V], br[CH][V];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int e = (i * TPR + t) * V;
        nv[i] = c - e < 0 ? 0 : (c - e < V ? c - e : V);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            wr[i][j] = w && j < nv[i] ? param(w, pdtype, e + j) : 1.0f;
            br[i][j] = b && j < nv[i] ? param(b, pdtype, e + j) : 0.0f;
        }
    }
    const float fc = (float)c;  // sums are divided, not scaled: a row of equal values has that very mean
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row0 = (int64_t)blockIdx.x * RPB;
    Raw16 next[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i)
        next[i] = load_raw(x + (row0 + g < n ? row0 + g : n - 1) * ldx + (i * TPR + t) * V, nv[i]);
    for (; row0 < n; row0 += step) {
        const int64_t row = row0 + g, ahead = row + step < n ? row + step : n - 1;
        float v[CH][V];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            unpack(next[i], v[i], x);
            if (row0 + step < n) next[i] = load_raw(x + ahead * ldx + (i * TPR + t) * V, nv[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) s += v[i][j];
        }
        const float mean = row_sum<TPR>(s, part, 0) / fc;
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] = nv[i] == V || j < nv[i] ? v[i][j] - mean : 0.0f;
                q += v[i][j] * v[i][j];
            }
        }
        const float r = rsqrtf(row_sum<TPR>(q, part, 1) / fc + eps);
        if (row < n) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
#pragma unroll
                for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * r * wr[i][j] + br[i][j];
                if (nv[i]) store_raw(y + row * ldy + (i * TPR + t) * V, repack(v[i], x), nv[i]);
            }
            if (stats && t == 0) stats[row] = make_float2(mean, r);
        }
    }
}

// dx, and each block's share of dw and db over its rows: kept in registers by the
// thread that owns the channel, summed over the block's row groups through LDS in a
// fixed order, written to partial [block][2][c] and summed over blocks by k_norm_wgrad; a
// single block writes dw and db itself (partial is NULL).  No atomics: the order is fixed.
// dx may be gy (so neither is restrict).
// 97,001 x 1024 bf16: 135 us for three passes over the rows, 4.4 TB/s, and 6 us for the sum.
template <typename T, int CH, int TPR>
__global__ __launch_bounds__(256) void k_norm_bwd(const T *gy, int64_t ldg, const T *__restrict__ x,
                                                  int64_t ldx, int64_t n, int c, const float2 *__restrict__ stats,
                                                  const void *__restrict__ w, int pdtype, T *dx,
                                                  int64_t lddx, float *__restrict__ partial, void *__restrict__ dw_out,
                                                  void *__restrict__ db_out)
{
    constexpr int V = VEC<T>, RPB = 256 / TPR, CPAD = CH * TPR * V;
    __shared__ float part[16];
    __shared__ __attribute__((aligned(16))) float red[RPB > 1 ? RPB * CPAD : 1];
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    int nv[CH];
    float wr[CH][V], dw[CH][V], db[CH][V];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int e = (i * TPR + t) * V;
        nv[i] = c - e < 0 ? 0 : (c - e < V ? c - e : V);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            wr[i][j] = w && j < nv[i] ? param(w, pdtype, e + j) : 1.0f;
            dw[i][j] = db[i][j] = 0.0f;
        }
    }
    const float fc = (float)c;  // sums are divided, not scaled: a row of equal values has that very mean
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row0 = (int64_t)blockIdx.x * RPB;
    Raw16 nx[CH], ng[CH];
    const int64_t first = row0 + g < n ? row0 + g : n - 1;
    float2 nst = stats[first];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        nx[i] = load_raw(x + first * ldx + (i * TPR + t) * V, nv[i]);
        ng[i] = load_raw(gy + first * ldg + (i * TPR + t) * V, nv[i]);
    }
    for (int k = 0; row0 < n; row0 += step, k ^= 1) {
        const int64_t row = row0 + g, ahead = row + step < n ? row + step : n - 1;
        const bool on = row < n;
        const float2 st = nst;
        float h[CH][V], gw[CH][V];
        float s1 = 0.0f, s2 = 0.0f;
        if (row0 + step < n) nst = stats[ahead];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            unpack(nx[i], h[i], x);
            unpack(ng[i], gw[i], x);
            if (row0 + step < n) {
                nx[i] = load_raw(x + ahead * ldx + (i * TPR + t) * V, nv[i]);
                ng[i] = load_raw(gy + ahead * ldg + (i * TPR + t) * V, nv[i]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {  // past the row's end g is zero, so h there adds nothing
                h[i][j] = (h[i][j] - st.x) * st.y;
                if (on) {
                    dw[i][j] += gw[i][j] * h[i][j];
                    db[i][j] += gw[i][j];
                }
                gw[i][j] *= wr[i][j];
                s1 += gw[i][j];
                s2 += gw[i][j] * h[i][j];
            }
        }
        s1 = row_sum<TPR>(s1, part, 2 * k) / fc;
        s2 = row_sum<TPR>(s2, part, 2 * k + 1) / fc;
        if (on) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] = st.y * (gw[i][j] - s1 - h[i][j] * s2);
                if (nv[i]) store_raw(dx + row * lddx + (i * TPR + t) * V, repack(h[i], x), nv[i]);
            }
        }
    }
    if (!partial && !dw_out && !db_out) return;
    float *mine = partial ? partial + (int64_t)blockIdx.x * 2 * c : nullptr;
    auto put = [&](int p, int e, float v) {
        if (mine) mine[p * c + e] = v;
        else set_param(p ? db_out : dw_out, pdtype, e, v);
    };
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if constexpr (RPB > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) red[g * CPAD + (i * TPR + t) * V + j] = p ? db[i][j] : dw[i][j];
            __syncthreads();
            for (int e = threadIdx.x; e < c; e += 256) {
                float s = 0.0f;
#pragma unroll 8
                for (int r = 0; r < RPB; ++r) s += red[r * CPAD + e];
                put(p, e, s);
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (j < nv[i]) put(p, (i * TPR + t) * V + j, p ? db[i][j] : dw[i][j]);
        }
    }
}

// dw and db: 16 columns of the partial sums a block, 16 threads to a column, then a
// sum over those in a fixed order.  No blocks (an empty set) leaves zeros.
__global__ __launch_bounds__(256) void k_norm_wgrad(const float *__restrict__ partial, int blocks, int c,
                                                    void *__restrict__ dw, void *__restrict__ db, int pdtype)
{
    __shared__ float red[16][17];
    const int col = blockIdx.x * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4;
    float s = 0.0f;
    if (col < 2 * c) {
#pragma unroll 8
        for (int b = part; b < blocks; b += 16) s += partial[(int64_t)b * 2 * c + col];
    }
    red[part][threadIdx.x & 15] = s;
    __syncthreads();
    if (part == 0 && col < 2 * c) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = red[i][threadIdx.x];
#pragma unroll
        for (int o = 8; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) v[i] += v[i + o];
        set_param(col < c ? dw : db, pdtype, col < c ? col : col - c, v[0]);
    }
}

// Threads a row and pieces a thread.  Up to 64 pieces of 16 bytes: the fewest lanes that
// hold the row, several rows to a wave; then a wave with up to 4 pieces a lane; then a
// block.
struct NormShape {
    int tpr, ch;
};
static NormShape norm_shape(int c, int dtype)
{
    const int v = dtype == SUBMCONV_F32 ? 4 : 8, pieces = (c + v - 1) / v;
    NormShape s = {64, 1};
    if (pieces <= 64) {
        s.tpr = 1;
        while (s.tpr < pieces) s.tpr *= 2;
    } else if (pieces <= 256) {
        s.ch = pieces <= 128 ? 2 : 4;
    } else {
        s.tpr = 256;
        s.ch = pieces <= 512 ? 2 : (pieces <= 1024 ? 4 : 8);
    }
    return s;
}

static int64_t norm_blocks(int64_t n, int c, int dtype, int64_t most)
{
    const int rows = 256 / norm_shape(c, dtype).tpr;
    const int64_t b = (n + rows - 1) / rows;
    return b < most ? b : most;
}

constexpr int64_t NORM_FWD_BLOCKS = 2048;  // eight to a compute unit
constexpr int64_t NORM_BWD_BLOCKS = 1024;
// Row groups that one block walks alone, to spare the second launch; where a row takes the whole
// block, only while the rows are few bytes too.  A call in us, two launches and one:
//   fp32, 8 groups:  x 16 17.4 and 13.6,  x 128 17.3 and 13.5,  x 1024 17.4 and 13.7
//   fp32, 32 groups: x 16 17.5 and 16.8,  x 128 17.3 and 17.0,  x 1024 17.4 and 44.4
//   fp32 x 2560:  6 rows 17.4 and 13.7,  12 rows 17.6 and 21.5
//   fp32 x 8192:  2 rows 17.4 and 14.9,  3 rows 17.5 and 19.2,  8 rows 17.6 and 41.0
//   bf16 x 8192:  4 rows 18.3 and 18.8,  8 rows 18.3 and 25.9
// Where the host does not set the pace (a replayed graph) the GPU's time counts, and the limit
// is near four groups (fp32 x 16: 5.2 and 4.7; 8 groups 5.3 and 6.4).
constexpr int64_t NORM_BWD_ALONE = 8, NORM_BWD_ALONE_BYTES = 64 << 10;

static int64_t norm_bwd_blocks(int64_t n, int c, int dtype)
{
    const int64_t b = norm_blocks(n, c, dtype, NORM_BWD_BLOCKS);
    const bool wide = norm_shape(c, dtype).tpr == 256;  // (then b rows in all)
    return b > 0 && b <= NORM_BWD_ALONE && (!wide || b * c * (dtype == SUBMCONV_F32 ? 4 : 2) <= NORM_BWD_ALONE_BYTES) ? 1 : b;
}

size_t norm_bwd_workspace(int64_t n, int c, int dtype)
{
    const int64_t blocks = norm_bwd_blocks(n, c, dtype);
    return blocks == 1 ? 0 : (size_t)blocks * 2 * c * sizeof(float);
}

#define NORM_SHAPES(T, GO)                                                         \
    switch (s.tpr * 16 + s.ch) {                                                   \
    case 1 * 16 + 1: GO(T, 1, 1); break;                                           \
    case 2 * 16 + 1: GO(T, 1, 2); break;                                           \
    case 4 * 16 + 1: GO(T, 1, 4); break;                                           \
    case 8 * 16 + 1: GO(T, 1, 8); break;                                           \
    case 16 * 16 + 1: GO(T, 1, 16); break;                                         \
    case 32 * 16 + 1: GO(T, 1, 32); break;                                         \
    case 64 * 16 + 1: GO(T, 1, 64); break;                                         \
    case 64 * 16 + 2: GO(T, 2, 64); break;                                         \
    case 64 * 16 + 4: GO(T, 4, 64); break;                                         \
    case 256 * 16 + 2: GO(T, 2, 256); break;                                       \
    case 256 * 16 + 4: GO(T, 4, 256); break;                                       \
    default:                                                                       \
        if constexpr (sizeof(T) == 4) GO(T, 8, 256);                               \
    }

int layer_norm(const void *x, int64_t ldx, int64_t n, int c, int dtype, const void *w, const void *b, int pdtype,
               float eps, void *y, int64_t ldy, float *stats, hipStream_t st)
{
    const NormShape s = norm_shape(c, dtype);
    const dim3 grid((unsigned)norm_blocks(n, c, dtype, NORM_FWD_BLOCKS));
#define GO(T, CH, TPR)                                                                                        \
    hipLaunchKernelGGL((k_norm<T, CH, TPR>), grid, dim3(256), 0, st, (const T *)x, ldx, n, c, w, b, pdtype,  \
                       eps, (T *)y, ldy, (float2 *)stats)
    if (dtype == SUBMCONV_F32) {
        NORM_SHAPES(float, GO)
    } else {
        NORM_SHAPES(uint16_t, GO)
    }
#undef GO
    SC_LAUNCHED("layer_norm");
    return SUBMCONV_OK;
}

int layer_norm_backward(const void *gy, int64_t ldg, const void *x, int64_t ldx, int64_t n, int c, int dtype,
                        const float *stats, const void *w, int pdtype, void *dx, int64_t lddx, void *dw, void *db,
                        void *workspace, hipStream_t st)
{
    const NormShape s = norm_shape(c, dtype);
    const int64_t blocks = norm_bwd_blocks(n, c, dtype);
    const bool alone = blocks == 1;
    float *partial = (dw || db) && !alone ? (float *)workspace : nullptr;
    if (n > 0) {
        const dim3 grid((unsigned)blocks);
#define GO(T, CH, TPR)                                                                                          \
    hipLaunchKernelGGL((k_norm_bwd<T, CH, TPR>), grid, dim3(256), 0, st, (const T *)gy, ldg, (const T *)x, ldx, \
                       n, c, (const float2 *)stats, w, pdtype, (T *)dx, lddx, partial, alone ? dw : nullptr,       \
                       alone ? db : nullptr)
        if (dtype == SUBMCONV_F32) {
            NORM_SHAPES(float, GO)
        } else {
            NORM_SHAPES(uint16_t, GO)
        }
#undef GO
        SC_LAUNCHED("layer_norm_backward");
    }
    if ((dw || db) && !alone) {
        hipLaunchKernelGGL(k_norm_wgrad, dim3((unsigned)((2 * c + 15) / 16)), dim3(256), 0, st, partial, (int)blocks,
                           c, dw, db, pdtype);
        SC_LAUNCHED("layer_norm_backward sums");
    }
    return SUBMCONV_OK;
}

}  // namespace sc
