// Rotation of head vectors by positions on several axes (a voxel's z, y, x).
//
// A head of `dim` elements is dim / 2 pairs.  Pair p belongs to an axis a(p) (the
// sections give each axis its run of pairs) and turns by t = position[a(p)] freq[p]:
//
//   (u, v) -> (u cos t - v sin t, u sin t + v cos t)
//
// Pairs past the last section stay as they are.  The inverse turns by -t; a rotation is
// orthogonal, so that is also its gradient.
//
// The kernel is bound by memory (each element read and written once).  A thread owns
// one 16-byte piece of the head (a piece of each half in the split layout), forms the
// sines and cosines of its pairs once and applies them to several heads of the row, four
// heads' loads in flight at a time.  400,311 x 24 x 128 bf16: 860 us, 5.7 TB/s (a plain
// device copy reaches 4.8 to 4.9); 20,384 x 24 x 128 inside a packed projection: 46 us, 5.5 TB/s.
#include "rotary.h"

namespace sc {

constexpr int64_t ROTARY_BLOCKS = 1 << 22;  // along x (a launch's axis holds 2^32 threads); the rest along y
constexpr int ROTARY_HEADS = 4;  // heads a thread works on at a time, their loads issued together

template <typename T, bool SPLIT>
__global__ __launch_bounds__(256) void k_rotary(const T *x, int64_t x_row, int64_t x_head,
                                                const int32_t *__restrict__ pos, int64_t pos_row,
                                                const float *__restrict__ freqs, RotaryAxes ax, int64_t n, int heads,
                                                int dim, int pieces, int hgroups, int rows_per_block, int inverse,
                                                T *out, int64_t out_row, int64_t out_head)
{
    constexpr int V = VEC<T>, PAIRS = SPLIT ? V : V / 2;
    const int per_row = pieces * hgroups;
    const int r = threadIdx.x / per_row, u = threadIdx.x - r * per_row;
    const int h0 = u / pieces, piece = u - h0 * pieces;
    const int64_t row = ((int64_t)blockIdx.y * ROTARY_BLOCKS + blockIdx.x) * rows_per_block + r;
    if (r >= rows_per_block || row >= n) return;

    const int half = dim / 2, used = ax.end[SUBMCONV_ROTARY_MAX_AXES - 1];
    const int e = piece * V;                      // first element (split: also first pair)
    const int left = (SPLIT ? half : dim) - e;
    const int nv = left < V ? left : V;
    const int turning = used - (SPLIT ? e : e / 2);  // pairs of the piece that turn; the others are copied as they are
    float c[PAIRS], s[PAIRS];
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
        const int p = (SPLIT ? e : e / 2) + j;
        c[j] = 1.0f;
        s[j] = 0.0f;
        if (p < used) {
            turn(pos[row * pos_row + rotary_axis(ax, p)], freqs[p], inverse != 0, &c[j], &s[j]);
        }
    }
    const T *xr = x + row * x_row + e;
    T *yr = out + row * out_row + e;
    for (int h = h0; h < heads; h += hgroups * ROTARY_HEADS) {
        Raw16 a[ROTARY_HEADS], b[ROTARY_HEADS];
#pragma unroll
        for (int i = 0; i < ROTARY_HEADS; ++i) {
            const int hh = h + i * hgroups;
            if (hh < heads) {
                a[i] = load_raw(xr + hh * x_head, nv);
                if (SPLIT) b[i] = load_raw(xr + hh * x_head + half, nv);
            }
        }
#pragma unroll
        for (int i = 0; i < ROTARY_HEADS; ++i) {
            const int hh = h + i * hgroups;
            if (hh >= heads) break;
            float va[V], vb[V];
            unpack(a[i], va, x);
            if constexpr (SPLIT) {
                unpack(b[i], vb, x);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float p = va[j], q = vb[j];
                    if (j >= turning) continue;
                    va[j] = p * c[j] - q * s[j];
                    vb[j] = p * s[j] + q * c[j];
                }
                store_raw(yr + hh * out_head + half, repack(vb, x), nv);
            } else {
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
                    const float p = va[2 * j], q = va[2 * j + 1];
                    if (j >= turning) continue;
                    va[2 * j] = p * c[j] - q * s[j];
                    va[2 * j + 1] = p * s[j] + q * c[j];
                }
            }
            store_raw(yr + hh * out_head, repack(va, x), nv);
        }
    }
}

int rotary(const void *x, int64_t x_row, int64_t x_head, const int32_t *pos, int64_t pos_row, const float *freqs,
           const int32_t *sections, int axes, int64_t n, int heads, int dim, int dtype, int split, int inverse,
           void *out, int64_t out_row, int64_t out_head, hipStream_t st)
{
    const RotaryAxes ax = rotary_axes(sections, axes);
    const int v = dtype == SUBMCONV_F32 ? 4 : 8, span = split ? dim / 2 : dim, pieces = (span + v - 1) / v;
    // one thread to a piece and ROTARY_HEADS heads while a block holds them
    int hgroups = (heads + ROTARY_HEADS - 1) / ROTARY_HEADS;
    if (hgroups * pieces > 256) hgroups = 256 / pieces;
    const int rows = 256 / (pieces * hgroups);
    const int64_t blocks = (n + rows - 1) / rows;
    const dim3 grid((unsigned)(blocks < ROTARY_BLOCKS ? blocks : ROTARY_BLOCKS), (unsigned)((blocks + ROTARY_BLOCKS - 1) / ROTARY_BLOCKS));
#define GO(T, SPLIT)                                                                                              \
    hipLaunchKernelGGL((k_rotary<T, SPLIT>), grid, dim3(256), 0, st, (const T *)x, x_row, x_head, pos, pos_row, freqs, \
                       ax, n, heads, dim, pieces, hgroups, rows, inverse, (T *)out, out_row, out_head)
    if (dtype == SUBMCONV_F32) {
        if (split) GO(float, true); else GO(float, false);
    } else {
        if (split) GO(uint16_t, true); else GO(uint16_t, false);
    }
#undef GO
    SC_LAUNCHED("rotary");
    return SUBMCONV_OK;
}

}  // namespace sc
