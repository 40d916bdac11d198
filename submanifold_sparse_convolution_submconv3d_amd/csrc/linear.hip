// Matrix products of ragged groups of rows, each with the weight of its group, and their gradients.
// For position i of group g, r = rows[i]:
//
//   y[i] = W_g x[r] + b_g,   dx[i] = W_g^T grad[i],   dW_g = sum over i in g of grad[i] x[r]^T,   db_g = sum grad[i]
//
// All three are products D[m, n] = sum over k of A[m, k] B[n, k]:
//
//        m            n      k          A                      B
//   y    positions    cout   cin        x, k next to each other    W_g, k next to each other
//   dx   positions    cin    cout       grad, k next to each other W_g, k a row apart
//   dW   cout         cin    positions  grad, k a row apart        x, k a row apart
//
// Sums are fp32; one rounding to the tensors' type at the end.  Every result element is summed by
// one lane in a fixed order, so the same call gives the same bits.
#include <type_traits>

#include "linear.h"

namespace sc {

constexpr int LT = 128;            // rows of either side in a tile
constexpr int LBYTES = 64 * LT;    // bytes of one side's tile for a step of 64 / sizeof(T) along k

// One side's tile in LDS.  Along k (KS false): rows of 64 bytes, their 16-byte pieces permuted so
// that 8 rows read at one piece fall on different banks.  Across k (KS true): 64 / sizeof(T)
// rows of LT elements; bf16 pieces are permuted for the transposing read, as in attention's tiles.
template <typename T, bool KS>
__device__ __forceinline__ uint32_t tile_at(uint32_t row, uint32_t piece)
{
    if constexpr (!KS) return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
    else if constexpr (sizeof(T) == 2) return piece_at<256>(row, piece);
    else return row * 512 + piece * 16;
}

// A lane's operand of a product of 32 rows from `block` on: its share of k step j (half of the tile's k).
template <typename T, bool KS>
__device__ __forceinline__ Raw16 tile_operand(uint32_t lds, int block, int j)
{
    const uint32_t l = lane_id(), a = l >> 5;
    if constexpr (!KS) {
        return lds_read16(lds + tile_at<T, KS>(block + (l & 31), 2 * j + a));
    } else if constexpr (sizeof(T) == 2) {
        // rows 16 j + 8 a + 4 h .. + 3 of k, transposed: lane t of 16 gets element t
        const uint32_t g = (l >> 4) & 1, t = l & 15, k = 16 * j + 8 * a + t / 4, piece = block / 8 + g * 2 + (t & 3) / 2;
        const u32x2 lo = lds_read_tr(lds + tile_at<T, KS>(k, piece) + (t & 1) * 8);
        const u32x2 hi = lds_read_tr(lds + tile_at<T, KS>(k + 4, piece) + (t & 1) * 8);
        return Raw16{lo[0], lo[1], hi[0], hi[1]};
    } else {
        Raw16 r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = *(const SC_LDS uint32_t *)(uintptr_t)(lds + (4 * (2 * j + a) + i) * 512 + (block + (l & 31)) * 4);
        return r;
    }
}

// Any widths, row distances and alignment: pieces of 16 bytes are loaded into registers with what
// is missing at the ends of rows as zeros, written to LDS, and the next step's loads are in flight
// meanwhile.  Four waves, each 64 x 64 of the tile.
// PART (LINEAR_DW): pieces of groups, whose sums are kept in fp32 for k_linear_join.
template <typename T, int KIND, bool PART>
__global__ __launch_bounds__(256) void k_linear(LinearArgs A)
{
    constexpr int V = VEC<T>, KT = 64 / (int)sizeof(T);
    constexpr bool AKS = KIND == LINEAR_DW, BKS = KIND != LINEAR_Y;
    __shared__ __attribute__((aligned(16))) char smem[4 * LBYTES];
    const uint32_t lds = (uint32_t)(uintptr_t)(SC_LDS char *)smem;
    const int wave = threadIdx.x >> 6;
    Part part;
    const int n_end = KIND == LINEAR_Y ? A.cout : A.cin;
    const uint32_t n_tiles = (n_end + LT - 1) / LT, other = blockIdx.x / n_tiles;
    int m0, m_end, n0 = (blockIdx.x - other * n_tiles) * LT, k_end;
    if constexpr (KIND == LINEAR_DW) {
        const uint32_t m_tiles = (A.cout + LT - 1) / LT, which = other / m_tiles;
        if constexpr (PART) {
            if (!find_tile(A, A.chunk, which, &part) || part.index < 1 || part.index > A.groups) return;
            part.beg += (int)part.tile * A.chunk;
            if (part.end - part.beg > A.chunk) part.end = part.beg + A.chunk;
        } else {
            group_bounds(A, which, &part);
        }
        m0 = (other - which * m_tiles) * LT;
        m_end = A.cout;
        k_end = part.end - part.beg;
    } else {
        if (!find_tile(A, LT, other, &part)) return;
        m0 = part.beg + (int)part.tile * LT;
        m_end = part.end;
        k_end = KIND == LINEAR_Y ? A.cin : A.cout;
    }
    const bool real = part.index >= 1 && part.index <= A.groups;
    const int group = real ? part.index - 1 : 0;
    if (!real) k_end = 0;  // rows of no group become zeros
    const T *w = (const T *)A.w + (int64_t)group * A.cout * A.cin;

    // A thread's two pieces of each side's tile.
    const T *a_row[2], *b_row[2];
    int r_[2][2], c_[2][2];  // row and first element of a piece in the tile
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = i * 256 + threadIdx.x;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const bool ks = s ? BKS : AKS;
            r_[s][i] = ks ? at / (LT / V) : at / 4;
            c_[s][i] = (ks ? at % (LT / V) : at % 4) * V;
        }
        if constexpr (!AKS) {
            const int p = m0 + r_[0][i];
            a_row[i] = nullptr;
            if (p < m_end) {
                if constexpr (KIND == LINEAR_DX) {
                    a_row[i] = (const T *)A.g + (int64_t)p * A.g_row;
                } else {
                    const int r = A.rows ? A.rows[p] : p;
                    if (r >= 0 && r < A.nx) a_row[i] = (const T *)A.x + (int64_t)r * A.x_row;
                }
            }
        }
        if constexpr (!BKS) b_row[i] = n0 + r_[1][i] < n_end ? w + (int64_t)(n0 + r_[1][i]) * A.cin : nullptr;
    }
    const auto left = [](int have) { return have < 0 ? 0 : (have < V ? have : V); };
    Raw16 av[2], bv[2];
    const auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            av[i] = bv[i] = Raw16{0, 0, 0, 0};
            if constexpr (!AKS) {
                const int nv = left(k_end - k0 - c_[0][i]);
                if (a_row[i] && nv) av[i] = load_raw(a_row[i] + k0 + c_[0][i], nv);
            } else {
                const int nv = left(m_end - m0 - c_[0][i]), k = k0 + r_[0][i];
                if (k < k_end && nv) av[i] = load_raw((const T *)A.g + (int64_t)(part.beg + k) * A.g_row + m0 + c_[0][i], nv);
            }
            if constexpr (!BKS) {
                const int nv = left(k_end - k0 - c_[1][i]);
                if (b_row[i] && nv) bv[i] = load_raw(b_row[i] + k0 + c_[1][i], nv);
            } else {
                const int nv = left(n_end - n0 - c_[1][i]), k = k0 + r_[1][i];
                if (k < k_end && nv) {
                    if constexpr (KIND == LINEAR_DX) {
                        bv[i] = load_raw(w + (int64_t)k * A.cin + n0 + c_[1][i], nv);
                    } else {
                        const int r = A.rows ? A.rows[part.beg + k] : part.beg + k;
                        if (r >= 0 && r < A.nx) bv[i] = load_raw((const T *)A.x + (int64_t)r * A.x_row + n0 + c_[1][i], nv);
                    }
                }
            }
        }
    };
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][0][e] = acc[i][1][e] = 0.0f;
    const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
    float sums[2] = {0.0f, 0.0f};  // db: of a lane's share of its rows of grad
    const bool summing = KIND == LINEAR_DW && A.db && n0 == 0 && wn == 0;
    load(0);
    for (int k0 = 0, buf = 0; k0 < k_end; k0 += KT, buf ^= 2 * LBYTES) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            lds_write16(lds + buf + tile_at<T, AKS>(r_[0][i], c_[0][i] / V), av[i]);
            lds_write16(lds + buf + LBYTES + tile_at<T, BKS>(r_[1][i], c_[1][i] / V), bv[i]);
        }
        __syncthreads();
        if (k0 + KT < k_end) load(k0 + KT);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            Raw16 a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = tile_operand<T, AKS>(lds + buf, wm + 32 * i, j);
                b[i] = tile_operand<T, BKS>(lds + buf + LBYTES, wn + 32 * i, j);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n) acc[m][n] = mma_pieces<T>(b[n], a[m], acc[m][n]);
            if (summing) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float v[V], t = 0.0f;
                    unpack(a[m], v, (const T *)nullptr);
#pragma unroll
                    for (int i = 0; i < V; i += 2) t += v[i] + v[i + 1];
                    sums[m] += t;
                }
            }
        }
    }
    // a lane has row l % 32 of each block, its elements in the registers
    const int l = lane_id() & 31;
    const int64_t ld = KIND == LINEAR_DW ? A.cin : A.out_row;
    typedef typename std::conditional<PART, float, T>::type Out;
    Out *out = PART ? (Out *)A.part : (Out *)A.out;
    const int64_t block = PART ? other / ((A.cout + LT - 1) / LT) : group;  // of dw
    if constexpr (KIND == LINEAR_DW) out += block * A.cout * A.cin;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int row = m0 + wm + 32 * m + l;
        const bool valid = row < m_end;
        if (summing) {
            const float sum = sums[m] + other_half(sums[m]);
            if (valid && lane_id() < 32) (PART ? A.db_part : A.db)[block * A.cout + row] = sum;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // registers 8h .. 8h + 3 and 8h + 4 .. 8h + 7: 8 elements in a row after the halves' exchange
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[m][n][8 * h + i]), __float_as_uint(acc[m][n][8 * h + 4 + i]), false, false);
                    v[i] = __uint_as_float(r[0]);
                    v[4 + i] = __uint_as_float(r[1]);
                }
                const int e = n0 + wn + 32 * n + 16 * h + 8 * (int)(lane_id() >> 5);
                if (!valid || e >= n_end) continue;
                if (KIND == LINEAR_Y && A.bias && real) {
                    const float *b = A.bias + (int64_t)group * A.cout + e;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (e + i < n_end) v[i] += b[i];
                }
                Out *to = out + (int64_t)row * ld + e;
                if constexpr (sizeof(Out) == 2) {
                    store_raw(to, repack(v, to), n_end - e < 8 ? n_end - e : 8);
                } else {
                    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
                    store_raw(to, repack(lo, to), n_end - e < 4 ? n_end - e : 4);
                    if (n_end - e > 4) store_raw(to + 4, repack(hi, to), n_end - e < 8 ? n_end - e - 4 : 4);
                }
            }
    }
}

// y for few rows a group (single tokens): bound by reading each weight once.  A block takes 16 positions and
// 16 NB columns; its four waves take a quarter of each run of k, with all their loads in flight, straight
// into the matrix instruction's operands (16 x 16, columns of y in the rows), and their sums are added in LDS.
template <typename T, int NB>
__global__ __launch_bounds__(256) void k_linear_few(LinearArgs A, int steps)
{
    constexpr int V = VEC<T>, KS = 4 * V, STEPS = 8;  // k of a step; most steps of a wave at a time
    __shared__ f32x4 part_sum[4][NB][64];
    const uint32_t cols = (A.cout + 16 * NB - 1) / (16 * NB), tile = blockIdx.x / cols;
    const int n0 = (int)(blockIdx.x - tile * cols) * 16 * NB, wave = threadIdx.x >> 6, l = (int)lane_id() & 15, q = (int)lane_id() >> 4;
    Part part;
    if (!find_tile(A, 16, tile, &part)) return;
    const bool real = part.index >= 1 && part.index <= A.groups;
    const int group = real ? part.index - 1 : 0, k_end = real ? A.cin : 0;
    const int p = part.beg + (int)part.tile * 16 + l;
    const T *w = (const T *)A.w + (int64_t)group * A.cout * A.cin, *wr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wr[b] = w + (int64_t)(n0 + 16 * b + l < A.cout ? n0 + 16 * b + l : A.cout - 1) * A.cin;
    int row = -1;
    if (p < part.end) row = A.rows ? A.rows[p] : p;
    const T *x = row >= 0 && row < A.nx ? (const T *)A.x + (int64_t)row * A.x_row : nullptr;
    f32x4 acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = f32x4{0, 0, 0, 0};
    for (int k0 = wave * steps * KS; k0 < k_end; k0 += 4 * steps * KS) {
        Raw16 wv[STEPS][NB], xv[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (s >= steps) break;
            const int k = k0 + s * KS + q * V, nv = k_end - k < 0 ? 0 : (k_end - k < V ? k_end - k : V);
#pragma unroll
            for (int b = 0; b < NB; ++b) wv[s][b] = load_raw(wr[b] + (nv ? k : 0), nv);
            xv[s] = x ? load_raw(x + (nv ? k : 0), nv) : Raw16{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (s >= steps) break;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if constexpr (sizeof(T) == 2) {
                    acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv[s][b]), __builtin_bit_cast(bf16x8, xv[s]), acc[b], 0, 0, 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(wv[s][b][i]), __uint_as_float(xv[s][i]), acc[b], 0, 0, 0);
                }
            }
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) part_sum[wave][b][lane_id()] = acc[b];
    __syncthreads();
    // a lane has position l % 16 and columns 4 (l / 16) .. + 3 of a block
    if (wave >= NB || p >= part.end) return;
    const f32x4 sum = (part_sum[0][wave][lane_id()] + part_sum[1][wave][lane_id()]) + (part_sum[2][wave][lane_id()] + part_sum[3][wave][lane_id()]);
    const int e = n0 + 16 * wave + 4 * q, have = A.cout - e;
    if (have <= 0) return;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = sum[i] + (A.bias && real && i < have ? A.bias[(int64_t)group * A.cout + e + i] : 0.0f);
    T *to = (T *)A.out + (int64_t)p * A.out_row + e;
    if constexpr (sizeof(T) == 4) {
        store_raw(to, repack(v, to), have < 4 ? have : 4);
    } else {
        const float eight[8] = {v[0], v[1], v[2], v[3], 0, 0, 0, 0};
        store_raw(to, repack(eight, to), have < 4 ? have : 4);
    }
}

// Sums of the pieces of each group, in order, rounded once; a block is 256 elements of a group's dw (and db).
template <typename T>
__global__ __launch_bounds__(256) void k_linear_join(LinearArgs A)
{
    const int64_t size = (int64_t)A.cout * A.cin, all = size + (A.db ? A.cout : 0), blocks = (all + 255) / 256;
    const int group = (int)(blockIdx.x / blocks);
    uint32_t first, count;
    group_tiles(A, A.chunk, group, &first, &count);
    const int64_t i = (blockIdx.x - group * blocks) * 256 + threadIdx.x;
    if (i >= all) return;
    const bool bias = i >= size;
    const float *from = bias ? A.db_part + (int64_t)first * A.cout + (i - size) : A.part + (int64_t)first * size + i;
    const int64_t step = bias ? A.cout : size;
    float sum = 0.0f;
#pragma unroll 8
    for (uint32_t p = 0; p < count; ++p) sum += from[p * step];
    if (bias) A.db[(int64_t)group * A.cout + (i - size)] = sum;
    else ((T *)A.out)[group * size + i] = Elem<T>::from_f32(sum);
}

// Positions of a piece of dw: whole groups (0) where these are blocks enough, else so many
// that the blocks of all pieces fill the card some times over.  A piece's sums are written and read again in
// fp32, so pieces are not shorter than 256 positions.
static int dw_chunk(int64_t n, int groups, int cin, int cout, bool big)
{
    const int size = big ? BIG_TILE : LT;
    const int64_t tiles = (int64_t)((cin + size - 1) / size) * ((cout + size - 1) / size), want = big ? UNITS : 4 * UNITS;
    if (groups * tiles >= want / 2 || n < 512) return 0;
    const int64_t pieces = (want + tiles - 1) / tiles;
    int64_t chunk = (n + pieces - 1) / pieces;
    chunk = (chunk + 63) / 64 * 64;
    return (int)(chunk < 256 ? 256 : chunk);
}

// Whether the large tiles may take a call of these widths.
static bool wide_enough(int cin, int cout, int dtype, int kind)
{
    return dtype == SUBMCONV_BF16 && cin % 8 == 0 && cout % 8 == 0 && (kind == LINEAR_Y ? cout : cin) >= 192 && (kind != LINEAR_DW || cout >= 192);
}

size_t linear_dw_workspace(int64_t n, int groups, int cin, int cout, int dtype)
{
    int64_t pieces = 0;
    for (int big = 0; big < 2; ++big) {
        if (big && !wide_enough(cin, cout, dtype, LINEAR_DW)) continue;
        const int chunk = dw_chunk(n, groups, cin, cout, big);
        const int64_t p = chunk ? most_tiles(n, groups, chunk) : 0;
        pieces = p > pieces ? p : pieces;
    }
    return (size_t)pieces * cout * ((size_t)cin + 1) * sizeof(float);
}

int64_t linear_blocks(int64_t n, int groups, int cin, int cout, int kind)
{
    return linear_tiles(n, groups, cin, cout, kind, kind == LINEAR_DW ? dw_chunk(n, groups, cin, cout, false) : 0, LT);
}

// Whether the large tiles take a call: bf16, whole pieces of 16 bytes everywhere, and both sides long
// enough.
static bool takes_big(const LinearArgs &A, int dtype, int kind)
{
    if (!wide_enough(A.cin, A.cout, dtype, kind)) return false;
    const auto pieces = [](const void *p, int64_t row) { return ((uintptr_t)p & 15) == 0 && row % 8 == 0; };
    if (kind != LINEAR_DX && !pieces(A.x, A.x_row)) return false;
    if (kind != LINEAR_Y && !pieces(A.g, A.g_row)) return false;
    if (kind != LINEAR_DW && !pieces(A.w, 0)) return false;
    return kind == LINEAR_DW || A.n / A.groups >= 128;
}

constexpr int64_t FEW_BLOCKS = 2048;
// Whether the kernel for few rows takes a call.
static bool takes_few(const LinearArgs &A)
{
    const int64_t blocks = most_tiles(A.n, A.groups, 16) * ((A.cout + 31) / 32);
    return blocks < 1 << 23 && (A.n <= 16 * (int64_t)A.groups || blocks <= FEW_BLOCKS);
}

int grouped_linear(LinearArgs A, int dtype, int kind, void *workspace, hipStream_t st)
{
    const bool big = takes_big(A, dtype, kind);
    if (kind == LINEAR_DW) {
        A.chunk = dw_chunk(A.n, A.groups, A.cin, A.cout, big);
        A.part = (float *)workspace;
        A.db_part = A.part + (A.chunk ? most_tiles(A.n, A.groups, A.chunk) * A.cout * A.cin : 0);
    }
    if (kind == LINEAR_Y && takes_few(A)) {
        constexpr int NB = 2;
        const int ks = dtype == SUBMCONV_F32 ? 16 : 32, quarter = (A.cin + 4 * ks - 1) / (4 * ks), steps = quarter < 8 ? quarter : 8;
        const dim3 grid((unsigned)(most_tiles(A.n, A.groups, 16) * ((A.cout + 16 * NB - 1) / (16 * NB))));
        if (dtype == SUBMCONV_F32) hipLaunchKernelGGL((k_linear_few<float, NB>), grid, dim3(256), 0, st, A, steps);
        else hipLaunchKernelGGL((k_linear_few<uint16_t, NB>), grid, dim3(256), 0, st, A, steps);
        SC_LAUNCHED("grouped_linear");
    } else if (big) {
        SC_CHECK(grouped_linear_big(A, kind, st));
    } else {
        const dim3 grid((unsigned)linear_tiles(A.n, A.groups, A.cin, A.cout, kind, A.chunk, LT));
#define GO(T, KIND, PART) hipLaunchKernelGGL((k_linear<T, KIND, PART>), grid, dim3(256), 0, st, A)
#define BY_KIND(T)                                 \
    if (kind == LINEAR_Y) GO(T, LINEAR_Y, false);  \
    else if (kind == LINEAR_DX) GO(T, LINEAR_DX, false); \
    else if (A.chunk) GO(T, LINEAR_DW, true);      \
    else GO(T, LINEAR_DW, false)
        if (dtype == SUBMCONV_F32) { BY_KIND(float); } else { BY_KIND(uint16_t); }
#undef BY_KIND
#undef GO
        SC_LAUNCHED("grouped_linear");
    }
    if (kind == LINEAR_DW && A.chunk) {
        const int64_t all = (int64_t)A.cout * A.cin + (A.db ? A.cout : 0);
        const dim3 grid((unsigned)((all + 255) / 256 * A.groups));
        if (dtype == SUBMCONV_F32) hipLaunchKernelGGL(k_linear_join<float>, grid, dim3(256), 0, st, A);
        else hipLaunchKernelGGL(k_linear_join<uint16_t>, grid, dim3(256), 0, st, A);
        SC_LAUNCHED("grouped_linear sums");
    }
    return SUBMCONV_OK;
}

}  // namespace sc
