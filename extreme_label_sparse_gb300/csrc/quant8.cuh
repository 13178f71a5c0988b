// Rows held in 8-bit integers: a group of columns (128, or the whole row) has a
// scale s = max |x| (1 / 127) and holds q = rint(x (127 (1 / max |x|))), each step
// in fp32; x is about q s.  Scales are at least 2^-126 (1 / s stays finite) and at most kMostScale, 0
// for a group of zeros, and NaN for a group that holds an infinity or NaN (its q
// are 0), so that such values are not lost silently.
#pragma once

#include "pairs.cuh"

namespace rows {

constexpr float kMostScale = 0x1.020406p+121f;  // the largest of which 127 are an fp32 number
constexpr int kGroup = 128;  // columns of a scale, where a row has several: half a warp's eights

struct Scale8 {
    float inv, scale;  // inv 0: not finite
};

// |v| as an integer that grows with it, infinities and NaN above all numbers
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The largest of eight magnitudes as mag() has it.  The 16-bit types compare two
// at a time, as they lie.
template <typename T>
__device__ __forceinline__ uint32_t top8(const Pack8<T> &p)
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&p);
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = max(m, w[j] & 0x7fffffffu);
        return m;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        const uint32_t h = max(m >> 16, m & 0xffffu);
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return h << 16;
        else
            return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
    }
}

__device__ __forceinline__ Scale8 scale8_of(uint32_t top)
{
    const float a = __uint_as_float(top);
    if (top >= 0x7f800000u)
        return {0.f, __uint_as_float(0x7fc00000u)};
    if (a < 127.0f * 0x1p-126f)
        return {0x1p126f, top ? 0x1p-126f : 0.f};
    return {__fmul_rn(__frcp_rn(a), 127.0f), fminf(__fmul_rn(a, 1.0f / 127.0f), kMostScale)};
}

// Eight values as int8.  Adding 1.5 2^23 rounds to whole numbers, ties to even,
// and leaves them in the sum's low bits; |v inv| stays below 127.5.
__device__ __forceinline__ uint2 quant8(const float2 (&v)[4], float inv)
{
    const float2 f = both(inv);
    float2 b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        b[i] = mul2(v[i], f);
        // one by one: as a pair the product and the sum were fused, and the
        // product lost its own rounding (other q where it falls on a half)
        b[i] = make_float2(__fadd_rn(b[i].x, 12582912.0f), __fadd_rn(b[i].y, 12582912.0f));
    }
    if (inv == 0.f)
        return make_uint2(0u, 0u);
    auto four = [](float2 x, float2 y) {
        return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                           __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
    };
    return make_uint2(four(b[0], b[1]), four(b[2], b[3]));
}

// Eight int8 as fp32: a byte plus 128 as the low bits of 2^23, less 2^23 + 128
// (conversions of integers run at a quarter of the rate).
__device__ __forceinline__ void unquant8(uint2 w, float2 (&v)[4])
{
    const float2 off = both(-8388736.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = (i < 2 ? w.x : w.y) ^ 0x80808080u;
        const int j = 2 * (i & 1);
        v[i] = add2(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 | j)),
                                __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 | (j + 1)))),
                    off);
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

// N segments of 256 columns (two groups each) to 8 bits, by all lanes of a warp:
// p are the lanes' eights, row(n), scale(n) and c0(n) the rows, their scales and
// the segments' first columns (a segment at or past `cols` is left out, as is one
// whose row is NULL).  The scales of all groups are worked out at once, by a lane
// each.
template <typename T, bool VEC, int N, typename Row, typename Scale, typename Col>
__device__ __forceinline__ void store_groups(const Pack8<T> (&p)[N], int lane, int cols, Row row, Scale scale, Col c0)
{
    static_assert(2 * N <= 16, "a lane of a half for each of its groups");
    uint32_t mine = 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if constexpr (VEC) {
            // half a warp has a group
            uint32_t top = top8(p[n]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if ((lane & 15) == n)
                mine = top;
        } else {
            // the first group is everybody's elements 0 to 3
            uint32_t a = 0, b = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a = max(a, mag(to_f(p[n].v[j])));
                b = max(b, mag(to_f(p[n].v[4 + j])));
            }
            a = __reduce_max_sync(0xffffffffu, a);
            b = __reduce_max_sync(0xffffffffu, b);
            if ((lane & 15) == n)
                mine = lane < 16 ? a : b;
        }
    }
    const Scale8 s = scale8_of(mine);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int at = c0(n) + (lane & 16) * 8;  // the group's first column
        if ((lane & 15) == n && row(n) && at < cols)
            scale(n)[at / kGroup] = s.scale;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float2 v[4];
        unpack4(p[n], v);
        uint2 w;
        if constexpr (VEC) {
            w = quant8(v, __shfl_sync(0xffffffffu, s.inv, (lane & 16) + n));
        } else {
            const float f = __shfl_sync(0xffffffffu, s.inv, n), g = __shfl_sync(0xffffffffu, s.inv, 16 + n);
            w = make_uint2(quant8(v, f).x, quant8(v, g).y);
        }
        if (row(n))
            store8q<VEC>(row(n), c0(n), lane, cols, w);
    }
}

// host: bytes of int8 rows can be taken in eights
inline bool vec8_ok(const void *p, int64_t ld) { return !p || (((uintptr_t)p) % 8 == 0 && ld % 8 == 0); }

}  // namespace rows
