// Rows of 16- and 32-bit floats as the row-wise operators read and write them
// (dropout, RMS norm), and the counter-based random bits of dropout.
//
// A warp takes segments of 256 columns of a row, eight elements to a lane.
// VEC: the lane's elements are contiguous; needs rows that start on eight
// elements' bytes and a whole number of eights.  Otherwise the lane takes
// columns lane, lane + 32, ...: any alignment and width, still whole sectors.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "sg_internal.cuh"
#include "tc_ptx.cuh"

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

// eight aligned elements: 16 bytes in one access; 32 (fp32) in two loads, which
// meet in L1, and one store, since halves of a sector would each go to L2
template <typename T>
__device__ __forceinline__ Pack8<T> load_pack(const T *src)
{
    Pack8<T> p;
#pragma unroll
    for (int i = 0; i < (int)sizeof(p) / 16; ++i)
        reinterpret_cast<uint4 *>(&p)[i] = reinterpret_cast<const uint4 *>(src)[i];
    return p;
}

template <typename T>
__device__ __forceinline__ void store_pack(T *dst, const Pack8<T> &p)
{
    if constexpr (sizeof(p) == 32)
        tc::st_global32(dst, reinterpret_cast<const uint32_t *>(&p));
    else
        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(&p);
}

// all eight at once: the 16-bit types convert in pairs
template <typename T>
__device__ __forceinline__ void unpack8(const Pack8<T> &p, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = to_f(p.v[j]);
}

template <typename T>
__device__ __forceinline__ Pack8<T> pack8(const float (&v)[8])
{
    Pack8<T> p;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p.v[j] = v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t &w = reinterpret_cast<uint32_t *>(&p)[j];
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
                w = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                w = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    return p;
}

// column of element j of this lane in the segment that starts at column c0
template <bool VEC>
__device__ __forceinline__ int col_of(int c0, int lane, int j)
{
    return VEC ? c0 + lane * 8 + j : c0 + lane + 32 * j;
}

// elements past `cols` read as zero
template <typename T, bool VEC>
__device__ __forceinline__ Pack8<T> load8(const T *row, int c0, int lane, int cols)
{
    Pack8<T> p;
    if constexpr (VEC) {
        if (c0 + lane * 8 < cols)
            return load_pack(row + c0 + lane * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p.v[j] = from_f<T>(0.f);
    } else {
        const T *at = row + c0 + lane;
        if (c0 + kSeg <= cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                p.v[j] = at[32 * j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                p.v[j] = col_of<VEC>(c0, lane, j) < cols ? at[32 * j] : from_f<T>(0.f);
        }
    }
    return p;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *row, int c0, int lane, int cols, const Pack8<T> &p)
{
    if constexpr (VEC) {
        if (c0 + lane * 8 < cols)
            store_pack(row + c0 + lane * 8, p);
    } else {
        T *at = row + c0 + lane;
        if (c0 + kSeg <= cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                at[32 * j] = p.v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col_of<VEC>(c0, lane, j) < cols)
                    at[32 * j] = p.v[j];
        }
    }
}

// ---------------------------------------------------------------- dropout
// What decides which elements stay: 16 random bits each, kept where they are
// at least `drop`; the kept ones are multiplied by 65536 / (65536 - drop).
struct Drop {
    uint32_t drop;  // 0 .. 65536; 0: no dropout
    uint32_t below;  // drop 2^16 - 1: a word is above it if its high half stays
    uint32_t c2, c3;
    float scale;
    // the keys of the ten rounds: the same for all threads, so they are worked
    // out once and read as constants
    uint32_t k0[10], k1[10];
};

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
// as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products.
__device__ __forceinline__ void philox10(const Drop &d, uint32_t x0, uint32_t x1, uint32_t (&w)[4])
{
    uint32_t x2 = d.c2, x3 = d.c3;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)x0 * 0xD2511F53u, q = (uint64_t)x2 * 0xCD9E8D57u;
        x0 = (uint32_t)(q >> 32) ^ x1 ^ d.k0[i];
        x1 = (uint32_t)q;
        x2 = (uint32_t)(p >> 32) ^ x3 ^ d.k1[i];
        x3 = (uint32_t)p;
    }
    w[0] = x0;
    w[1] = x1;
    w[2] = x2;
    w[3] = x3;
}

// Which of a lane's eight elements of a segment stay.  VEC: they are the eight
// of one block, and the block's random words are looked at as they are;
// without it an element's bits come from the lane that drew its block, so
// every lane of the warp makes one.  drop is not 0.
template <bool VEC>
struct Keep {
    uint32_t w[VEC ? 4 : 1];
    uint32_t below;

    __device__ __forceinline__ Keep(const Drop &d, int c0, int lane, uint32_t row)
    {
        uint32_t r[4];
        philox10(d, (uint32_t)(c0 / 8) + lane, row, r);
        below = d.below;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = r[i];
        } else {
            uint32_t own = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                own |= (r[i] << 16 > below ? 1u : 0u) << (2 * i);
                own |= (r[i] > below ? 1u : 0u) << (2 * i + 1);
            }
            w[0] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[0] |= ((__shfl_sync(0xffffffffu, own, (lane >> 3) + 4 * j) >> (lane & 7)) & 1u) << j;
        }
    }

    __device__ __forceinline__ bool at(int j) const
    {
        if constexpr (VEC)
            return ((j & 1) ? w[j / 2] : w[j / 2] << 16) > below;
        else
            return (w[0] >> j) & 1u;
    }
};

// host: the fields of Drop, false if p is not a probability
inline bool make_drop(double p, uint64_t seed, uint64_t offset, Drop *d)
{
    if (!(p >= 0.0 && p <= 1.0))
        return false;
    d->drop = (uint32_t)(p * 65536.0 + 0.5);
    d->below = (uint32_t)(((uint64_t)d->drop << 16) - 1);
    d->c2 = (uint32_t)offset;
    d->c3 = (uint32_t)(offset >> 32);
    for (uint32_t i = 0; i < 10; ++i) {
        d->k0[i] = (uint32_t)seed + i * 0x9E3779B9u;
        d->k1[i] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
    }
    // at drop = 65536 nothing is kept and the factor is not used
    d->scale = d->drop < 65536u ? (float)(65536.0 / (double)(65536u - d->drop)) : 0.f;
    return true;
}

// host: a matrix can be taken in pieces of eight elements (a NULL one does not
// hinder)
inline bool vec_ok(const void *p, int64_t ld, int64_t elem)
{
    return !p || (((uintptr_t)p) % (8 * elem) == 0 && ld % 8 == 0);
}

}  // namespace rows
