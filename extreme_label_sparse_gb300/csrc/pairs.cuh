// fp32 arithmetic on pairs (one instruction for two elements), and eights of
// 16-bit and 32-bit floats as four of them.
#pragma once

#include "rows.cuh"

namespace rows {

__device__ __forceinline__ uint64_t bits2(float2 a)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 pair2(uint64_t r)
{
    float2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return pair2(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

template <typename T>
__device__ __forceinline__ void unpack4(const Pack8<T> &p, float2 (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(&p)[i];
            v[i] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        } else if constexpr (std::is_same<T, __half>::value) {
            v[i] = __half22float2(reinterpret_cast<const __half2 *>(&p)[i]);
        } else {
            v[i] = make_float2(p.v[2 * i], p.v[2 * i + 1]);
        }
    }
}

template <typename T>
__device__ __forceinline__ Pack8<T> pack4(const float2 (&v)[4])
{
    const float e[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    return pack8<T>(e);
}

}  // namespace rows
