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
// one lane in a fixed order (or by a few whose sums are added in a fixed order), so the same call gives the same bits.
//
// Here: tiles of 64 and 128 for any alignment and for calls of middling size, and a kernel for few rows; linear_big.hip
// has the large tiles.  Offsets are read on the device; a block finds its tile from them.
#include <type_traits>

#include "linear.h"

namespace sc {

// Tiles of 64 B rows of either side, in steps of KB bytes along k: 64 x 64 in steps of 128 bytes, 128 x 128 in
// steps of 64.  A thread has two pieces of 16 bytes of each side's tile.
template <typename T, int B>
struct TileShape {
    static constexpr int LT = 64 * B, KB = 128 / B, KT = KB / (int)sizeof(T), BYTES = LT * KB;
};

// One side's tile in LDS.  Along k (KS false): rows of KB bytes.  Across k (KS true): KT rows of LT
// elements.  Pieces are permuted as in attention's tiles, but for fp32 across k, which is read by elements.
template <typename T, int B, bool KS>
__device__ __forceinline__ uint32_t tile_at(uint32_t row, uint32_t piece)
{
    using S = TileShape<T, B>;
    if constexpr (!KS) return piece_at<S::KB>(row, piece);
    else if constexpr (sizeof(T) == 2) return piece_at<S::LT * 2>(row, piece);
    else return row * (S::LT * 4) + piece * 16;
}

// A lane's operand of a product of 32 rows from `block` on: its share of 32 bytes of k, number j of the step.
template <typename T, int B, bool KS>
__device__ __forceinline__ Raw16 tile_operand(uint32_t lds, int block, int j)
{
    const uint32_t l = lane_id(), a = l >> 5;
    if constexpr (!KS) {
        return lds_read16(lds + tile_at<T, B, KS>(block + (l & 31), 2 * j + a));
    } else if constexpr (sizeof(T) == 2) {
        // rows 16 j + 8 a + 4 h .. + 3 of k, transposed: lane t of 16 gets element t
        const uint32_t g = (l >> 4) & 1, t = l & 15, k = 16 * j + 8 * a + t / 4, piece = block / 8 + g * 2 + (t & 3) / 2;
        const u32x2 lo = lds_read_tr(lds + tile_at<T, B, KS>(k, piece) + (t & 1) * 8);
        const u32x2 hi = lds_read_tr(lds + tile_at<T, B, KS>(k + 4, piece) + (t & 1) * 8);
        return Raw16{lo[0], lo[1], hi[0], hi[1]};
    } else {
        Raw16 r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = *(const SC_LDS uint32_t *)(uintptr_t)(lds + (4 * (2 * j + a) + i) * (TileShape<T, B>::LT * 4) + (block + (l & 31)) * 4);
        return r;
    }
}

// Any widths, row distances and alignment: pieces of 16 bytes are loaded into registers a step or two ahead and
// written to LDS, with what is missing at the ends of rows as zeros.  Four waves, each a quarter of the tile.
// Loads without branches are what counts: with one at each row's end the compiler waited for every load before the next
// (3 x 3000 rows of 1001 -> 999 in fp32, y, dx, dw with db: 211, 253, 318 us; without, in tiles of 64, 64 and 128, 175, 191, 226, 103
// to 80 TFLOP/s.  The rules below take tiles of 128 there: 212, 226, 226; bf16 61, 50, 75).
// 20,384 rows of 123 -> 501 in fp32: 44, 42, 47 us and 8 for the pieces' sums, where 17 is the matrix cores' time: one
// or two rounds of short blocks, whose first loads and last stores nothing covers, and unaligned 16-byte accesses.
// Weights that few rows share are read at the memory's rate: 8 x 1 rows of 1024 -> 4096 in bf16 13.0 us for 67 MB.
// PART (LINEAR_DW): pieces of groups, whose sums are kept in fp32 for k_linear_join.
// SHORT: rows may be shorter than a piece, and are loaded by elements.
template <typename T, int KIND, bool PART, int B, bool SHORT>
__global__ __launch_bounds__(256) void k_linear(LinearArgs A)
{
    using S = TileShape<T, B>;
    constexpr int V = VEC<T>, KT = S::KT, LT = S::LT, BYTES = S::BYTES;
    constexpr bool AKS = KIND == LINEAR_DW, BKS = KIND != LINEAR_Y;
    __shared__ __attribute__((aligned(16))) char smem[4 * BYTES];
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
            r_[s][i] = ks ? at / (LT / V) : at / (S::KB / 16);
            c_[s][i] = (ks ? at % (LT / V) : at % (S::KB / 16)) * V;
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
    constexpr int AHEAD = B == 1 ? 2 : 1;  // steps that loads run ahead (more registers cost the large tiles a block a compute unit)
    Raw16 av_[AHEAD][2], bv_[AHEAD][2];
    // elements from `at` on of a row of `end`
    const auto load_piece = [&](const T *row, int at, int end) {
        if constexpr (SHORT) {
            return row && at < end ? load_raw(row + at, end - at < V ? end - at : V) : Raw16{0, 0, 0, 0};
        } else {
            const T *p = row + (at < end - V ? at : end - V);
            return load_global(row && at < end ? p : (const T *)zero_piece);
        }
    };
    int x_rows[2] = {0, 0};  // LINEAR_DW: of the next step, loaded a step ahead
    const auto look_up = [&](int k0) {
        if constexpr (KIND == LINEAR_DW) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int p = part.beg + k0 + r_[1][i];
                x_rows[i] = p < A.n ? p : A.n - 1;
            }
            if (A.rows && A.n) {
#pragma unroll
                for (int i = 0; i < 2; ++i) x_rows[i] = A.rows[x_rows[i]];
            }
        }
    };
    const auto load = [&](int k0, Raw16 (&av)[2], Raw16 (&bv)[2]) {
        const int r_now[2] = {x_rows[0], x_rows[1]};
        look_up(k0 + KT);  // (first: a wait for these is a wait for what was loaded before them too)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ka = k0 + r_[0][i], kb = k0 + r_[1][i];
            if constexpr (!AKS) av[i] = load_piece(a_row[i], k0 + c_[0][i], k_end);
            else av[i] = load_piece(ka < k_end ? (const T *)A.g + (int64_t)(part.beg + ka) * A.g_row : nullptr, m0 + c_[0][i], m_end);
            if constexpr (!BKS) bv[i] = load_piece(b_row[i], k0 + c_[1][i], k_end);
            else if constexpr (KIND == LINEAR_DX) bv[i] = load_piece(kb < k_end ? w + (int64_t)kb * A.cin : nullptr, n0 + c_[1][i], n_end);
            else bv[i] = load_piece(kb < k_end && r_now[i] >= 0 && r_now[i] < A.nx ? (const T *)A.x + (int64_t)r_now[i] * A.x_row : nullptr, n0 + c_[1][i], n_end);
        }
    };
    // What was loaded of before the rows' ends is dropped, in the tiles and steps that have some.
    const auto drop_ends = [&](int k0, Raw16 (&av)[2], Raw16 (&bv)[2]) {
        if constexpr (SHORT) return;
        if (AKS ? m0 + LT > m_end : k0 + KT > k_end)
#pragma unroll
            for (int i = 0; i < 2; ++i) av[i] = drop(av[i], AKS ? past<V>(m0 + c_[0][i], m_end) : past<V>(k0 + c_[0][i], k_end), (const T *)nullptr);
        if (BKS ? n0 + LT > n_end : k0 + KT > k_end)
#pragma unroll
            for (int i = 0; i < 2; ++i) bv[i] = drop(bv[i], BKS ? past<V>(n0 + c_[1][i], n_end) : past<V>(k0 + c_[1][i], k_end), (const T *)nullptr);
    };
    const int wm = (wave & 1) * (32 * B), wn = (wave >> 1) * (32 * B), half = (int)lane_id() >> 5;
    f32x16 acc[B][B];  // a lane has row l % 32 of each block, its elements in the registers
    float sums[B];  // db: of a lane's share of its rows of grad
#pragma unroll
    for (int i = 0; i < B; ++i) sums[i] = 0.0f;
    const bool summing = KIND == LINEAR_DW && A.db && n0 == 0 && wn == 0;
    const auto step = [&](int k0, int buf, Raw16 (&av)[2], Raw16 (&bv)[2]) {
        drop_ends(k0, av, bv);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            lds_write16(lds + buf + tile_at<T, B, AKS>(r_[0][i], c_[0][i] / V), av[i]);
            lds_write16(lds + buf + BYTES + tile_at<T, B, BKS>(r_[1][i], c_[1][i] / V), bv[i]);
        }
        __syncthreads();
        load(k0 + AHEAD * KT, av, bv);  // zeros past the end: a load that may not be there costs a wait for all
        Raw16 a_[2][B], b_[2][B];
        const auto read = [&](int j) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
                a_[j % 2][i] = tile_operand<T, B, AKS>(lds + buf, wm + 32 * i, j);
                b_[j % 2][i] = tile_operand<T, B, BKS>(lds + buf + BYTES, wn + 32 * i, j);
            }
        };
        read(0);
#pragma unroll
        for (int j = 0; j < S::KB / 32; ++j) {
            Raw16 (&a)[B] = a_[j % 2], (&b)[B] = b_[j % 2];
            if (j + 1 < S::KB / 32) read(j + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < B; ++m)
#pragma unroll
                for (int n = 0; n < B; ++n) acc[m][n] = mma_pieces<T>(b[n], a[m], acc[m][n]);
            if (summing) {
#pragma unroll
                for (int m = 0; m < B; ++m) {
                    float v[V], t = 0.0f;
                    unpack(a[m], v, (const T *)nullptr);
#pragma unroll
                    for (int i = 0; i < V; i += 2) t += v[i] + v[i + 1];
                    sums[m] += t;
                }
            }
        }
    };
    look_up(0);
    load(0, av_[0], bv_[0]);
    if constexpr (AHEAD == 2) load(KT, av_[1], bv_[1]);
    // sums begin with the bias
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
        for (int n = 0; n < B; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][n][e] = 0.0f;
    if (KIND == LINEAR_Y && A.bias && real) {
        const float *bias = A.bias + (int64_t)group * A.cout;
#pragma unroll
        for (int n = 0; n < B; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = n0 + wn + 32 * n + 8 * (i / 4) + 4 * half + i % 4;
                const float v = bias[e < n_end ? e : n_end - 1];
#pragma unroll
                for (int m = 0; m < B; ++m) acc[m][n][i] = v;
            }
    }
    if constexpr (AHEAD == 2) {
        for (int k0 = 0; k0 < k_end; k0 += 2 * KT) {
            step(k0, 0, av_[0], bv_[0]);
            if (k0 + KT < k_end) step(k0 + KT, 2 * BYTES, av_[1], bv_[1]);
        }
    } else {
        for (int k0 = 0, buf = 0; k0 < k_end; k0 += KT, buf ^= 2 * BYTES) step(k0, buf, av_[0], bv_[0]);
    }
    const int l = lane_id() & 31;
    const int64_t ld = KIND == LINEAR_DW ? A.cin : A.out_row;
    typedef typename std::conditional<PART, float, T>::type Out;
    Out *out = PART ? (Out *)A.part : (Out *)A.out;
    const int64_t block = PART ? other / ((A.cout + LT - 1) / LT) : group;  // of dw
    if constexpr (KIND == LINEAR_DW) out += block * A.cout * A.cin;
#pragma unroll
    for (int m = 0; m < B; ++m) {
        const int row = m0 + wm + 32 * m + l;
        const bool valid = row < m_end;
        if (summing) {
            const float sum = sums[m] + other_half(sums[m]);
            if (valid && lane_id() < 32) (PART ? A.db_part : A.db)[block * A.cout + row] = sum;
        }
#pragma unroll
        for (int n = 0; n < B; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // registers 8h .. 8h + 3 and 8h + 4 .. 8h + 7: 8 elements in a row after the halves' exchange
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[m][n][8 * h + i]), __float_as_uint(acc[m][n][8 * h + 4 + i]), false, false);
                    v[i] = __uint_as_float(r[0]);
                    v[4 + i] = __uint_as_float(r[1]);
                }
                const int e = n0 + wn + 32 * n + 16 * h + 8 * half;
                if (!valid || e >= n_end) continue;
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

// y for few rows a group (single tokens): bound by reading each weight once, or by the launch (450 x 2 rows of 64 -> 256
// in fp32: 5.2 us; tiles of 64 take as long there, but 25 instead of 8 where 1024 of k are walked by few blocks).  A block takes 16 positions and
// 16 NB columns; its four waves take a quarter of each run of k, with all their loads in flight, straight
// into the matrix instruction's operands (16 x 16, columns of y in the rows), and their sums are added in LDS.
template <typename T, int NB, bool SHORT>
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
            const int k = k0 + s * KS + q * V;
            const auto load_piece = [&](const T *row) {
                if constexpr (SHORT) {
                    return row && k < k_end ? load_raw(row + k, k_end - k < V ? k_end - k : V) : Raw16{0, 0, 0, 0};
                } else {
                    const T *p = row + (k < k_end - V ? k : k_end - V);
                    return load_global(row && k < k_end ? p : (const T *)zero_piece);
                }
            };
#pragma unroll
            for (int b = 0; b < NB; ++b) wv[s][b] = load_piece(wr[b]);
            xv[s] = load_piece(x);
        }
        if (!SHORT && k0 + steps * KS > k_end) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (s >= steps) break;
                const int over = past<V>(k0 + s * KS + q * V, k_end);
#pragma unroll
                for (int b = 0; b < NB; ++b) wv[s][b] = drop(wv[s][b], over, (const T *)nullptr);
                xv[s] = drop(xv[s], over, (const T *)nullptr);
            }
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

// The rules below were measured over 1 to 8 groups of 1 to 8192 rows, widths of 61 to 4096, in us a call; what they compare
// is the blocks or tiles of a call, n cols, and n cin cout.  (Rows a group are not looked at.)
//   y, few rows (16 a tile) and tiles of 64, bf16: 8 groups of 1024 -> 4096, 1 row each, 16.6 and 13.0 (640 tiles of 64);
//     3 x 64 x 1001 -> 999 17.0 and 10.4 (544 blocks of few); fp32: 1 x 256 x 1024 -> 1024 17.7 and 25.5 (608),
//     8 x 32 x 1024 -> 1024 18.2 and 25.7 (832), 64 rows 31.7 and 26.1 (1344), 5 x 512 x 501 -> 123 13.8 and 15.0 (668).
//   y, tiles of 64 and the ring of 128, bf16: 8 x 64 x 1024 -> 1024 10.4 and 14.9, 256 rows 12.8 and 15.3, 512 19.6 and 17.0;
//     dx, 8 x 64 x 1024 -> 4096 31.7 and 40.1; fp32: 8 x 256 x 1024 -> 1024 44 and 76, 512 rows 79 and 78;
//     dx, 8 x 8192 x 64 -> 256 32.2 and 41.8 (half of a tile of 128 is empty; the rule for widths below 96 has tiles of 128
//     through registers there, 43).
//   y and dx, the rings of 128 and 256, bf16: 8 x 512 x 1024 -> 1024 17 and 29, 8 x 2048 43 and 37, 8 x 8192 167 and 135.
//   y and dx, tiles of 64 and 128 (unaligned), bf16: 3 x 1024 x 1001 -> 999 23.9 and 31.4 (192 tiles of 128), 8 x 512 x 255 ->
//     1023 14.6 and 13.4 (256), dx 3 x 2048 x 1001 -> 999 41.9 and 33.8 (384); fp32: 8 x 4096 x 255 -> 1023 184 and 174 (2048),
//     dx 176 and 157 (512), but 3 x 3000 x 1001 -> 999 175 and 212 (560).
//   dw, tiles of 64 and 128, bf16: 5 x 4096 x 123 x 501 31.0 and 25.5 (1.3e9 products), 8 x 32 x 1024 x 1024 13.4 and 13.4 (512
//     tiles); fp32: 5 x 8192 x 123 x 501 87 and 79 (2.5e9), 8 x 32 x 1024 x 1024 17.4 and 15.0 (512 tiles);
//     tiles of 128 and the ring of 256, bf16: 8 x 256 x 1024 x 1024 14.0 and 19.2 (2.1e9); 8 x 8192 x 256 x 256 47.4 and 38.8, 4 x 4096
//     x 512 x 512 43.6 and 37.2, 64 x 256 x 512 x 512 26.2 and 20.3 (4.3e9 each), 8 x 2048 x 1024 x 4096 216 and 146 (6.9e10).  Where
//     whole groups leave half of the card idle tiles of 128 are faster, which products alone do not show: 8 x 512 x 1024 x 1024
//     21.2 and 27.5, 2048 rows 64 and 68, 4096 rows 122 and 124;
//     tiles of 128 and the ring of 128, fp32: 8 x 128 x 1024 x 1024 29.1 and 28.8 (1.1e9), 8 x 256 48.3 and 46.2.
constexpr int64_t FEW_ROWS = 16, BIG_OUT = 1 << 24, RING_OUT = 1 << 22;
constexpr int64_t few_blocks(bool f32) { return f32 ? 1024 : 512; }  // at most, for few rows
constexpr int64_t few_tiles(bool f32) { return f32 ? INT64_MAX : 512; }  // of 64, up to FEW_ROWS a group
constexpr int64_t large_tiles(bool f32) { return f32 ? 512 : 288; }  // of 128 from here on, ends of groups not counted
constexpr double ring_dw(bool f32) { return f32 ? 2e9 : 4e9; }
constexpr double large_dw(bool f32) { return f32 ? 2e9 : 1.2e9; }

// Which kernel takes a call.
enum { BY_FEW, BY_SMALL, BY_LARGE, BY_RING, BY_BIG };  // (the last two: linear_big.hip)
constexpr int TILE_OF[] = {16, 64, 128, 128, 256};

// Positions of a piece of dw: whole groups (0) where these are blocks enough, else so many
// that the blocks of all pieces fill the card some times over.  A piece's sums are written and read again in
// fp32, so pieces are not shorter than 256 positions.
static int dw_chunk(int64_t n, int groups, int cin, int cout, int by)
{
    const int size = TILE_OF[by];
    const int64_t tiles = (int64_t)((cin + size - 1) / size) * ((cout + size - 1) / size), want = UNITS * (by == BY_BIG ? 1 : (by == BY_RING ? 2 : (by == BY_LARGE ? 4 : 16)));
    if (groups * tiles >= want / 2 || n < 512) return 0;
    const int64_t pieces = (want + tiles - 1) / tiles;
    int64_t chunk = (n + pieces - 1) / pieces;
    chunk = (chunk + 63) / 64 * 64;
    return (int)(chunk < 256 ? 256 : chunk);
}

// Whether the ring kernels may take a call of these widths, if pointers and distances are aligned.
static bool may_be_big(int cin, int cout, int dtype)
{
    const int v = dtype == SUBMCONV_F32 ? 4 : 8;
    return cin % v == 0 && cout % v == 0;
}

// Whether rows may have less than a piece of 16 bytes.
static bool is_short(int cin, int cout, int dtype)
{
    const int v = dtype == SUBMCONV_F32 ? 4 : 8;
    return cin < v || cout < v;
}

// The kernel by sizes alone; `aligned`: whole pieces of 16 bytes everywhere.
static int choose(int64_t n, int groups, int cin, int cout, int dtype, int kind, bool aligned)
{
    const int cols = kind == LINEAR_Y ? cout : cin;
    const bool f32 = dtype == SUBMCONV_F32, ring = aligned && may_be_big(cin, cout, dtype);
    if (kind == LINEAR_Y) {
        const int64_t blocks = most_tiles(n, groups, 16) * ((cout + 31) / 32);
        if (blocks <= few_blocks(f32) || (n <= FEW_ROWS * (int64_t)groups && linear_tiles(n, groups, cin, cout, kind, 0, 64) <= few_tiles(f32))) return BY_FEW;
    }
    if (is_short(cin, cout, dtype)) return BY_SMALL;
    const double work = (double)n * cin * cout;
    if (kind == LINEAR_DW) {
        if (ring && work >= ring_dw(f32) && cin >= 96 && cout >= 96 && (f32 || (cin >= 192 && cout >= 192))) return f32 ? BY_RING : BY_BIG;
        return work >= large_dw(f32) || linear_tiles(n, groups, cin, cout, kind, 0, 128) >= 512 ? BY_LARGE : BY_SMALL;
    }
    if (ring && !f32 && n * cols >= BIG_OUT && cols >= 192) return BY_BIG;
    if (ring && n * cols >= RING_OUT && cols >= 96) return BY_RING;
    return n / 128 * ((cols + 127) / 128) >= large_tiles(f32) ? BY_LARGE : BY_SMALL;
}

size_t linear_dw_workspace(int64_t n, int groups, int cin, int cout, int dtype)
{
    int64_t pieces = 0;
    for (int aligned = 0; aligned < 2; ++aligned) {
        const int chunk = dw_chunk(n, groups, cin, cout, choose(n, groups, cin, cout, dtype, LINEAR_DW, aligned));
        const int64_t p = chunk ? most_tiles(n, groups, chunk) : 0;
        pieces = p > pieces ? p : pieces;
    }
    return (size_t)pieces * cout * ((size_t)cin + 1) * sizeof(float);
}

// Blocks of a call whose tensors are not aligned (aligned ones take as many or fewer).
int64_t linear_blocks(int64_t n, int groups, int cin, int cout, int dtype, int kind)
{
    const int by = choose(n, groups, cin, cout, dtype, kind, false);
    if (by == BY_FEW) return most_tiles(n, groups, 16) * ((cout + 31) / 32);
    return linear_tiles(n, groups, cin, cout, kind, kind == LINEAR_DW ? dw_chunk(n, groups, cin, cout, by) : 0, TILE_OF[by]);
}

static bool is_aligned(const LinearArgs &A, int dtype, int kind)
{
    const int v = dtype == SUBMCONV_F32 ? 4 : 8;
    const auto pieces = [&](const void *p, int64_t row) { return ((uintptr_t)p & 15) == 0 && row % v == 0; };
    if (kind != LINEAR_DX && !pieces(A.x, A.x_row)) return false;
    if (kind != LINEAR_Y && !pieces(A.g, A.g_row)) return false;
    return kind == LINEAR_DW || pieces(A.w, 0);
}

int grouped_linear(LinearArgs A, int dtype, int kind, void *workspace, hipStream_t st)
{
    const int by = choose(A.n, A.groups, A.cin, A.cout, dtype, kind, is_aligned(A, dtype, kind));
    if (kind == LINEAR_DW) {
        A.chunk = dw_chunk(A.n, A.groups, A.cin, A.cout, by);
        A.part = (float *)workspace;
        A.db_part = A.part + (A.chunk ? most_tiles(A.n, A.groups, A.chunk) * A.cout * A.cin : 0);
    }
    if (by == BY_FEW) {
        constexpr int NB = 2;
        const int ks = dtype == SUBMCONV_F32 ? 16 : 32, quarter = (A.cin + 4 * ks - 1) / (4 * ks), steps = quarter < 8 ? quarter : 8;
        const dim3 grid((unsigned)(most_tiles(A.n, A.groups, 16) * ((A.cout + 16 * NB - 1) / (16 * NB))));
#define GO(T)                                                                                                   \
    if (A.cin < VEC<T>) hipLaunchKernelGGL((k_linear_few<T, NB, true>), grid, dim3(256), 0, st, A, steps);      \
    else hipLaunchKernelGGL((k_linear_few<T, NB, false>), grid, dim3(256), 0, st, A, steps)
        if (dtype == SUBMCONV_F32) { GO(float); } else { GO(uint16_t); }
#undef GO
        SC_LAUNCHED("grouped_linear");
    } else if (by >= BY_RING) {
        SC_CHECK(grouped_linear_big(A, dtype, kind, TILE_OF[by], st));
    } else {
        const dim3 grid((unsigned)linear_tiles(A.n, A.groups, A.cin, A.cout, kind, A.chunk, TILE_OF[by]));
        const bool by_elements = is_short(A.cin, A.cout, dtype);  // (never in tiles of 128)
#define GO(T, KIND, PART)                                                                                                  \
    if (by_elements) hipLaunchKernelGGL((k_linear<T, KIND, PART, 1, true>), grid, dim3(256), 0, st, A);     \
    else if (by == BY_SMALL) hipLaunchKernelGGL((k_linear<T, KIND, PART, 1, false>), grid, dim3(256), 0, st, A);           \
    else hipLaunchKernelGGL((k_linear<T, KIND, PART, 2, false>), grid, dim3(256), 0, st, A)
#define BY_KIND(T)                                              \
    if (kind == LINEAR_Y) { GO(T, LINEAR_Y, false); }           \
    else if (kind == LINEAR_DX) { GO(T, LINEAR_DX, false); }    \
    else if (A.chunk) { GO(T, LINEAR_DW, true); }               \
    else { GO(T, LINEAR_DW, false); }
        if (dtype == SUBMCONV_F32) { BY_KIND(float) } else { BY_KIND(uint16_t) }
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
