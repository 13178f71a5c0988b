// Rows of 16- and 32-bit floats as the row-wise operators read and write them
// (dropout, RMS norm), and the counter-based random bits of dropout.
//
// A warp takes segments of 256 columns of a row, eight elements to a lane.
// VEC: the lane's elements are contiguous (16-byte accesses); needs rows that
// start on 16 bytes and a whole number of eights.  Otherwise the lane takes
// columns lane, lane + 32, ...: any alignment and width, still whole sectors.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sg_internal.cuh"

namespace rows {

constexpr int kSeg = 256;  // columns of a warp's segment

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f(float v) { return v; }

// eight elements as they lie in memory
template <typename T>
struct alignas(16) Pack8 {
    T v[8];
};

// column of element j of this lane in the segment that starts at column c0
template <bool VEC>
__device__ __forceinline__ int64_t col_of(int64_t c0, int lane, int j)
{
    return VEC ? c0 + lane * 8 + j : c0 + lane + 32 * j;
}

// elements past `cols` read as zero
template <typename T, bool VEC>
__device__ __forceinline__ Pack8<T> load8(const T *row, int64_t c0, int lane, int64_t cols)
{
    Pack8<T> p;
    if constexpr (VEC) {
        if (c0 + lane * 8 < cols) {
            const uint4 *src = reinterpret_cast<const uint4 *>(row + c0 + lane * 8);
#pragma unroll
            for (int i = 0; i < (int)sizeof(p) / 16; ++i)
                reinterpret_cast<uint4 *>(&p)[i] = src[i];
            return p;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p.v[j] = from_f<T>(0.f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = col_of<VEC>(c0, lane, j);
            p.v[j] = c < cols ? row[c] : from_f<T>(0.f);
        }
    }
    return p;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *row, int64_t c0, int lane, int64_t cols, const Pack8<T> &p)
{
    if constexpr (VEC) {
        if (c0 + lane * 8 < cols) {
            uint4 *dst = reinterpret_cast<uint4 *>(row + c0 + lane * 8);
#pragma unroll
            for (int i = 0; i < (int)sizeof(p) / 16; ++i)
                dst[i] = reinterpret_cast<const uint4 *>(&p)[i];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = col_of<VEC>(c0, lane, j);
            if (c < cols)
                row[c] = p.v[j];
        }
    }
}

// ---------------------------------------------------------------- dropout
// What decides which elements stay: 16 random bits each, kept where they are
// at least `drop`; the kept ones are multiplied by 65536 / (65536 - drop).
struct Drop {
    uint32_t drop;  // 0 .. 65536; 0: no dropout
    uint32_t k0, k1, c2, c3;
    float scale;
};

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
// as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products.
__device__ __forceinline__ uint4 philox10(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, uint32_t k0,
                                          uint32_t k1)
{
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)x0 * 0xD2511F53u, q = (uint64_t)x2 * 0xCD9E8D57u;
        x0 = (uint32_t)(q >> 32) ^ x1 ^ k0;
        x1 = (uint32_t)q;
        x2 = (uint32_t)(p >> 32) ^ x3 ^ k1;
        x3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

// bit j: element j of the eight columns 8 blk .. 8 blk + 7 of `row` stays
__device__ __forceinline__ uint32_t keep8(const Drop &d, uint32_t blk, uint32_t row)
{
    const uint4 r = philox10(blk, row, d.c2, d.c3, d.k0, d.k1);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m |= ((w[i] & 0xffffu) >= d.drop ? 1u : 0u) << (2 * i);
        m |= ((w[i] >> 16) >= d.drop ? 1u : 0u) << (2 * i + 1);
    }
    return m;
}

// the same for this lane's elements of a segment (every lane of the warp calls
// it: without VEC an element's bits come from the lane of its block)
template <bool VEC>
__device__ __forceinline__ uint32_t keep_lane(const Drop &d, int64_t c0, int lane, uint32_t row)
{
    const uint32_t own = keep8(d, (uint32_t)(c0 / 8 + lane), row);
    if constexpr (VEC)
        return own;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        m |= ((__shfl_sync(0xffffffffu, own, (lane >> 3) + 4 * j) >> (lane & 7)) & 1u) << j;
    return m;
}

// host: the fields of Drop, false if p is not a probability
inline bool make_drop(double p, uint64_t seed, uint64_t offset, Drop *d)
{
    if (!(p >= 0.0 && p <= 1.0))
        return false;
    d->drop = (uint32_t)(p * 65536.0 + 0.5);
    d->k0 = (uint32_t)seed;
    d->k1 = (uint32_t)(seed >> 32);
    d->c2 = (uint32_t)offset;
    d->c3 = (uint32_t)(offset >> 32);
    // at drop = 65536 nothing is kept and the factor is not used
    d->scale = d->drop < 65536u ? (float)(65536.0 / (double)(65536u - d->drop)) : 0.f;
    return true;
}

// host: a matrix can be taken in 16-byte pieces (a NULL one does not hinder)
inline bool vec_ok(const void *p, int64_t ld, int64_t elem)
{
    return !p || ((((uintptr_t)p) & 15) == 0 && (ld * elem) % 16 == 0);
}

}  // namespace rows
