// What the 8-bit linear layer's kernels share: its status word, and int8 rows in 16
// bits.
#pragma once

#include "launch.cuh"
#include "quant8.cuh"
#include "tc_tile.cuh"

namespace {

#define LIN_FAIL(code, ...)        \
    do {                           \
        sg_set_error(__VA_ARGS__); \
        return code;               \
    } while (0)
#define LIN_TRY(expr)           \
    do {                        \
        sg_status rc_ = (expr); \
        if (rc_ != SG_OK)       \
            return rc_;         \
    } while (0)

constexpr int kSMs = 152;

// errors of calls that were given no status word
__device__ int32_t g_linear_status;

__device__ __forceinline__ int32_t *lin_status(int32_t *status) { return status ? status : &g_linear_status; }

// two of four int8 (bytes 0 and 1, or 2 and 3 of u ^ 0x80808080) as fp16, by the
// usual way of 8-bit weights on 16-bit tensor cores: a byte plus 128 as the low bits
// of 1024, less 1152
__device__ __forceinline__ uint32_t bytes_f16(uint32_t u, int half)
{
    const uint32_t h = __byte_perm(u, 0x64646464u, half ? 0x4342 : 0x4140);
    const __half2 v =
        __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half((unsigned short)0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 16 bytes at column c (a whole number of 16) of a row of `cols`, 0 past the last;
// vec: the row starts on 16 bytes
__device__ __forceinline__ void bytes16(const int8_t *row, int c, int cols, bool vec, uint32_t (&in)[4])
{
    if (vec && c + 16 <= cols) {
        *reinterpret_cast<uint4 *>(in) = *reinterpret_cast<const uint4 *>(row + c);
    } else if (c + 16 <= cols) {
        // rows that start anywhere: the words that the bytes lie in
        const int off = (int)((uintptr_t)(row + c) & 3);
        const uint32_t *at = reinterpret_cast<const uint32_t *>(row + c - off);
        const uint32_t end = off ? at[4] : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            in[j] = at[j];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            in[j] = __funnelshift_r(in[j], j < 3 ? in[j + 1] : end, 8 * off);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            in[j] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + 4 * j + k < cols)
                    in[j] |= (uint32_t)(uint8_t)row[c + 4 * j + k] << (8 * k);
        }
    }
}

// int8 rows that do not start on 16 bytes, copied to rows that do, of a whole
// number of 16 (0 past the last column): 48 bytes of traffic for 16, where bringing
// them to 16 bits takes 80.  A warp takes a row, or 512 columns of one where there
// are few rows.
__global__ void __launch_bounds__(256)
    k_realign(const int8_t *__restrict__ src, int64_t ld, int64_t rows, int cols, int spans, int8_t *__restrict__ dst,
              int64_t ldd)
{
    const int lane = threadIdx.x & 31;
    grid_wait();
    grid_go();
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; i < rows * spans; i += (int64_t)gridDim.x * 8) {
        const int64_t r = spans > 1 ? i / spans : i;
        const int first = spans > 1 ? (int)(i - r * spans) * 512 : 0, last = spans > 1 ? min(cols, first + 512) : cols;
#pragma unroll 4
        for (int c = first + lane * 16; c < last; c += 512) {
            uint32_t in[4];
            bytes16(src + r * ld, c, cols, false, in);
            *reinterpret_cast<uint4 *>(dst + r * ldd + c) = make_uint4(in[0], in[1], in[2], in[3]);
        }
    }
}

// A power of two that brings the largest of n scales to about [256, 512), where the
// largest magnitude held in 8 bits (128 times it) is still an fp16 number, and its
// inverse: for all THREADS of a CTA.  fp16 rounds 65520 to infinity, so a scale
// that would come to 511.875 or more is brought to half of that.
template <int THREADS>
__device__ __forceinline__ float2 factor_of(const float *s, int64_t n, float *sm)
{
    float top = 0.f;
    // eight under way together; those past the end read the last again
    for (int64_t i = threadIdx.x; i < n; i += 8 * THREADS) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = fabsf(s[min(i + j * THREADS, n - 1)]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = fmaxf(top, v[j] < INFINITY ? v[j] : 0.f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        sm[threadIdx.x / 32] = top;
    __syncthreads();
    for (int i = 0; i < THREADS / 32; ++i)
        top = fmaxf(top, sm[i]);
    int e = 0;
    if (top > 0.f) {
        const float f = frexpf(top, &e);  // top = f 2^e, f in [1/2, 1)
        e = (f < 511.875f / 512.0f ? 9 : 8) - e;
    }
    e = e > 126 ? 126 : e;
    return make_float2(ldexpf(1.f, e), ldexpf(1.f, -e));
}

struct Widen {
    const int8_t *src;
    int64_t ld, rows;
    int32_t cols, group;   // group: columns of a scale, 0: the row's
    const float *scale;    // NULL: the integers themselves, in fp16
    float *factor;         // of the scales, and its inverse, or NULL
    int32_t scales;        // if not 0: the factor is not there yet, and goes by so many
    uint16_t *dst;
    int64_t ldd;           // a whole number of 16
    int32_t f16, vec;      // vec: rows start on 16 bytes
    int32_t spans;         // of a row, a warp each
};

// int8 rows to 16 bits: the integers, or the values they stand for, of one or two
// matrices.  The gradients' sums run over what the scales belong to, so a scale has to
// enter a product's operand; the value is rounded to dout's type there, as 16-bit weights
// would be (two operands for its high and low bits would double the products: dx and
// dW are off by 2.4e-3 in bf16 so, 1.7e-3 without).  A warp takes a row, or a span of one where there are few, 16 columns
// to a lane, whose 32 bytes it writes at once (halves of a sector would each go to L2: 64 MB took 40 us).
__global__ void __launch_bounds__(256) k_widen(const __grid_constant__ Widen m0, const __grid_constant__ Widen m1)
{
    const int lane = threadIdx.x & 31;
    grid_wait();
    grid_go();
    // few scales: each CTA works the factors out, one keeps them for later launches
    __shared__ float sm[8];
    float2 f0 = make_float2(1.f, 1.f), f1 = f0;
    if (m0.scales)
        f0 = factor_of<256>(m0.scale, m0.scales, sm);
    else if (m0.factor)
        f0.x = *m0.factor;
    if (m1.scales)
        f1 = factor_of<256>(m1.scale, m1.scales, sm);
    else if (m1.factor)
        f1.x = *m1.factor;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (m0.scales)
            *reinterpret_cast<float2 *>(m0.factor) = f0;
        if (m1.scales)
            *reinterpret_cast<float2 *>(m1.factor) = f1;
    }
    const int64_t n0 = m0.rows * m0.spans, n = n0 + m1.rows * m1.spans;
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; i < n; i += (int64_t)gridDim.x * 8) {
        const bool second = i >= n0;
        const Widen &a = second ? m1 : m0;
        int64_t r = second ? i - n0 : i;
        int first = 0, last = a.cols;
        if (a.spans > 1) {
            const int64_t u = r;
            r = u / a.spans;
            first = (int)(u - r * a.spans) * 512;
            last = min(a.cols, first + 512);
        }
        const int ng = a.group ? (a.cols + a.group - 1) / a.group : 1;
        const float f = second ? f1.x : f0.x;
        const int8_t *src = a.src + r * a.ld;
        const float *sc = a.scale ? a.scale + r * ng : nullptr;
        uint16_t *dst = a.dst + r * a.ldd;
#pragma unroll 4
        for (int c = first + lane * 16; c < last; c += 512) {
            uint32_t in[4];
            bytes16(src, c, a.cols, a.vec, in);
            uint32_t w[8];
            if (!sc) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = bytes_f16(in[j / 2] ^ 0x80808080u, j & 1);
            } else {
                // a group is a whole number of 16 columns
                const float s = sc[a.group ? c / a.group : 0] * f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float2 v[4];
                    rows::unquant8(make_uint2(in[2 * k], in[2 * k + 1]), v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j] = rows::mul2(v[j], rows::both(s));
                        w[4 * k + j] = pack16(v[j].x, v[j].y, a.f16);
                    }
                }
            }
            st_global32(dst + c, w);
        }
    }
}

// ---------------------------------------------------------------- host
Widen widen_of(const int8_t *src, int64_t ld, int64_t rows, int64_t cols, const float *scale, int32_t group,
               float *factor, uint8_t *dst, int64_t ldd, bool f16, int64_t scales = 0)
{
    const bool vec = ((uintptr_t)src & 15) == 0 && ld % 16 == 0;
    return {src,    ld,  rows, (int32_t)cols, group, scale, factor, (int32_t)scales, reinterpret_cast<uint16_t *>(dst),
            ldd, f16, vec,  1};
}

// after: as launch() has it
sg_status widen(Widen a, Widen b, bool after, cudaStream_t st)
{
    const int64_t most = kSMs * 8;
    // few rows: a warp to 512 columns (128 x 2048: 3 us less)
    const bool few = a.rows + b.rows < 2 * most;
    a.spans = few ? (int32_t)ceil_div(a.cols, 512) : 1;
    b.spans = few ? (int32_t)ceil_div(b.cols, 512) : 1;
    const int64_t need = ceil_div(a.rows * a.spans + b.rows * b.spans, 8);
    return launch(k_widen, dim3((unsigned)(need < most ? need : most)), 256, 0, 1, after, st, a, b);
}

sg_status realign(const int8_t *src, int64_t ld, int64_t rows, int64_t cols, uint8_t *dst, int64_t ldd, bool after,
                  cudaStream_t st)
{
    const int64_t most = kSMs * 8, spans = rows < 2 * most ? ceil_div(cols, 512) : 1, need = ceil_div(rows * spans, 8);
    return launch(k_realign, dim3((unsigned)(need < most ? need : most)), 256, 0, 1, after, st, src, ld, rows, (int)cols,
                  (int)spans, reinterpret_cast<int8_t *>(dst), ldd);
}

}  // namespace
