// Rows held in 8-bit integers: a group of columns (128, or the whole row) has a
// scale s = max |x| / 127 and holds q = rint(x (127 / max |x|)); x is about q s.
// Scales are at least 2^-126 (1 / s stays finite) and at most kMostScale, 0 for a
// group of zeros, and NaN for a group that holds an infinity or NaN (its q are
// 0), so that such values are not lost silently.
#pragma once

#include "rows.cuh"

namespace rows {

constexpr float kMostScale = 0x1.020406p+121f;  // the largest of which 127 are an fp32 number
constexpr int kGroup = 128;  // columns of a scale, where a row has several: half a warp's eights

struct Scale8 {
    float inv, scale;  // inv 0: not finite
};

// |v| as an integer that grows with it, infinities and NaN above all numbers
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ Scale8 scale8_of(uint32_t top)
{
    const float a = __uint_as_float(top);
    if (top >= 0x7f800000u)
        return {0.f, __uint_as_float(0x7fc00000u)};
    if (a < 127.0f * 0x1p-126f)
        return {0x1p126f, top ? 0x1p-126f : 0.f};
    return {__fdiv_rn(127.0f, a), fminf(__fdiv_rn(a, 127.0f), kMostScale)};
}

// Eight values as int8.  Adding 1.5 2^23 rounds to whole numbers, ties to even,
// and leaves them in the sum's low bits; |v inv| stays below 127.5.
__device__ __forceinline__ uint2 quant8(const float (&v)[8], float inv)
{
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        b[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.0f));
    if (inv == 0.f)
        return make_uint2(0u, 0u);
    uint2 w;
    w.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    w.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    return w;
}

__device__ __forceinline__ void unquant8(uint2 w, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = (float)(int8_t)(w.x >> (8 * j));
        v[4 + j] = (float)(int8_t)(w.y >> (8 * j));
    }
}

// A lane's eight bytes of a segment (see col_of); bytes past `cols` read as 0
// and are not written.
template <bool VEC>
__device__ __forceinline__ uint2 load8q(const int8_t *row, int c0, int lane, int cols)
{
    uint2 w = make_uint2(0u, 0u);
    if constexpr (VEC) {
        if (c0 + lane * 8 < cols)
            w = *reinterpret_cast<const uint2 *>(row + c0 + lane * 8);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = col_of<false>(c0, lane, j);
            const uint32_t b = c < cols ? (uint32_t)(uint8_t)row[c] : 0u;
            (j < 4 ? w.x : w.y) |= b << (8 * (j & 3));
        }
    }
    return w;
}

template <bool VEC>
__device__ __forceinline__ void store8q(int8_t *row, int c0, int lane, int cols, uint2 w)
{
    if constexpr (VEC) {
        if (c0 + lane * 8 < cols)
            *reinterpret_cast<uint2 *>(row + c0 + lane * 8) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = col_of<false>(c0, lane, j);
            if (c < cols)
                row[c] = (int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
        }
    }
}

// A warp's segment of 256 columns (two groups) to 8 bits, by all of its lanes;
// `row` and `scale` are the row's.
template <bool VEC>
__device__ __forceinline__ void store_groups(int8_t *row, float *scale, int c0, int lane, int cols,
                                             const float (&v)[8])
{
    if constexpr (VEC) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, mag(v[j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const Scale8 s = scale8_of(top);
        if ((lane & 15) == 0 && c0 + lane * 8 < cols)
            scale[c0 / kGroup + lane / 16] = s.scale;
        store8q<VEC>(row, c0, lane, cols, quant8(v, s.inv));
    } else {
        // the first group is everybody's elements 0 to 3
        uint32_t a = 0, b = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a = max(a, mag(v[j]));
            b = max(b, mag(v[4 + j]));
        }
        const Scale8 s = scale8_of(__reduce_max_sync(0xffffffffu, a)), t = scale8_of(__reduce_max_sync(0xffffffffu, b));
        if (lane == 0) {
            if (c0 < cols)
                scale[c0 / kGroup] = s.scale;
            if (c0 + kGroup < cols)
                scale[c0 / kGroup + 1] = t.scale;
        }
        store8q<VEC>(row, c0, lane, cols, make_uint2(quant8(v, s.inv).x, quant8(v, t.inv).y));
    }
}

// the eight values that a lane's bytes of a segment stand for
template <bool VEC>
__device__ __forceinline__ void load_groups(const int8_t *row, const float *scale, int c0, int lane, int cols,
                                            float (&v)[8])
{
    unquant8(load8q<VEC>(row, c0, lane, cols), v);
    if constexpr (VEC) {
        const float s = c0 + lane * 8 < cols ? scale[c0 / kGroup + lane / 16] : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= s;
    } else {
        const float s = c0 < cols ? scale[c0 / kGroup] : 0.f, t = c0 + kGroup < cols ? scale[c0 / kGroup + 1] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] *= s;
            v[4 + j] *= t;
        }
    }
}

// host: bytes of int8 rows can be taken in eights
inline bool vec8_ok(const void *p, int64_t ld) { return !p || (((uintptr_t)p) % 8 == 0 && ld % 8 == 0); }

}  // namespace rows
