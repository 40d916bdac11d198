// Row pieces of 16 bytes and sums over groups of lanes, shared by the kernels that
// stream feature rows (norm.hip, rotary.hip).
#pragma once

#include "common.h"

namespace sc {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 16 bytes of a row at any element address: gfx950 loads and stores them with one
// instruction whatever the alignment, so odd widths and offsets take the same path.
typedef uint32_t Raw16 __attribute__((ext_vector_type(4)));
typedef uint32_t Raw16Any __attribute__((ext_vector_type(4), aligned(2)));

template <typename T> constexpr int VEC = 16 / (int)sizeof(T);

// Two fp32 values rounded to bf16 (nearest even, NaN stays NaN) in one word.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ void unpack(const Raw16 &r, float (&v)[4], const float *)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void unpack(const Raw16 &r, float (&v)[8], const uint16_t *)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ Raw16 repack(const float (&v)[4], const float *)
{
    Raw16 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]);
    return r;
}
__device__ __forceinline__ Raw16 repack(const float (&v)[8], const uint16_t *)
{
    Raw16 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    return r;
}

// The first nv elements at p (nv <= VEC), the rest zero.
__device__ __forceinline__ Raw16 load_raw(const float *p, int nv)
{
    Raw16 r = {0, 0, 0, 0};
    if (nv == 4) return *(const Raw16Any *)p;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < nv) r[i] = __float_as_uint(p[i]);
    return r;
}
__device__ __forceinline__ Raw16 load_raw(const uint16_t *p, int nv)
{
    Raw16 r = {0, 0, 0, 0};
    if (nv == 8) return *(const Raw16Any *)p;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < nv) r[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    return r;
}
__device__ __forceinline__ void store_raw(float *p, const Raw16 &r, int nv)
{
    if (nv == 4) {
        *(Raw16Any *)p = r;
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < nv) p[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void store_raw(uint16_t *p, const Raw16 &r, int nv)
{
    if (nv == 8) {
        *(Raw16Any *)p = r;
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < nv) p[i] = (uint16_t)(r[i / 2] >> (16 * (i & 1)));
}

// Sum over aligned groups of L lanes (a power of two up to 64), the same bits in every
// lane: each step adds the two halves of a group in either order.  The lanes of a group
// must all be active.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    if constexpr (L >= 2) v = dpp_add<0xb1>(v);    // lane ^ 1 within a quad
    if constexpr (L >= 4) v = dpp_add<0x4e>(v);    // lane ^ 2
    if constexpr (L >= 8) v = dpp_add<0x141>(v);   // the other quad of 8 (mirrored: quads hold one value)
    if constexpr (L >= 16) v = dpp_add<0x140>(v);  // the other half of 16
    if constexpr (L >= 32) {
        auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (L >= 64) {
        auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

}  // namespace sc
