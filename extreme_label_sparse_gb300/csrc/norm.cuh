// What the norms' kernels and the other operators on whole rows share: a row in
// the registers of a CTA, its sums, the next rows on their way to shared memory,
// the join of the column sums, and the checks of arguments.
#pragma once

#include <atomic>

#include "launch.cuh"
#include "rows.cuh"

using namespace rows;

namespace {

#define NORM_FAIL(code, ...)       \
    do {                           \
        sg_set_error(__VA_ARGS__); \
        return code;               \
    } while (0)

#define NORM_TRY(expr)          \
    do {                        \
        sg_status rc_ = (expr); \
        if (rc_ != SG_OK)       \
            return rc_;         \
    } while (0)

constexpr int64_t kMaxCols = 32768;   // of the norm: a row lies in one CTA's registers
constexpr int kSMs = 152;

// Sum of a (and, if MAX, maximum of b) over the WARPS warps of a row group (all of
// the CTA where WARPS > 1).  Every thread gets both.  Successive calls take turns
// with two buffers, so that one barrier is enough.
struct RowSums {
    float2 v[2][32];
};

template <int WARPS, bool MAX>
__device__ __forceinline__ void row_reduce(float &a, float &b, RowSums &sm, int turn)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        if (MAX)
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    if constexpr (WARPS > 1) {
        if ((threadIdx.x & 31) == 0)
            sm.v[turn & 1][threadIdx.x / 32] = make_float2(a, b);
        __syncthreads();
        // a lane takes a warp's values, and the shuffles above once more
        const float2 t = sm.v[turn & 1][threadIdx.x % WARPS];
        a = t.x;
        b = t.y;
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            if (MAX)
                b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
    }
}

// A thread's pieces of the next rows on their way to shared memory: NA
// matrices, NV pieces of eight elements each, S rows deep.  Each thread copies
// (cp.async) exactly what it reads itself, so no barrier is needed, and rows
// in flight take no registers.
template <typename T, int NA, int NV, int S, int THREADS>
struct Ring8 {
    static constexpr int kPieces = sizeof(Pack8<T>) / 16;
    static constexpr int kBytes = S * NA * NV * kPieces * THREADS * 16;
    uint4 *base;

    __device__ __forceinline__ explicit Ring8(void *smem) : base(static_cast<uint4 *>(smem) + threadIdx.x) {}
    __device__ __forceinline__ uint4 *at(int slot, int m, int n, int i) const
    {
        return base + (((slot * NA + m) * NV + n) * kPieces + i) * THREADS;
    }
    __device__ __forceinline__ void copy(int slot, int m, int n, const T *src) const
    {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t dst = tc::smem_u32(at(slot, m, n, i));
            if constexpr (kPieces == 2)
                tc::cp_async16_l1(dst, reinterpret_cast<const uint4 *>(src) + i);
            else
                tc::cp_async16(dst, reinterpret_cast<const uint4 *>(src) + i);
        }
    }
    __device__ __forceinline__ Pack8<T> get(int slot, int m, int n) const
    {
        Pack8<T> p;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            reinterpret_cast<uint4 *>(&p)[i] = *at(slot, m, n, i);
        return p;
    }
};

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// threads of a CTA, and CTAs to an SM that the registers are cut for: 1024
// threads of 64 registers, or 512 of 128
constexpr int norm_threads(int warps) { return warps == 1 ? 256 : warps * 32; }
constexpr int norm_ctas(int warps, bool few)
{
    const int n = (few ? 512 : 1024) / norm_threads(warps);
    return n < 1 ? 1 : n;
}

// dweight[c] = the sum of its parts, in a fixed order: NC columns to a CTA,
// whose threads take 1024 / NC parts at a time.  Eight columns (a sector) give
// enough CTAs where there are few columns (65536 x 256, whole backward pass: 32
// us, 37 with 32 columns), 32 read whole lines (16384 x 4096: 123 us, 125).
template <int NC>
__global__ void __launch_bounds__(1024) k_norm_dw(const float *__restrict__ part, int nparts, int64_t cols,
                                                  float *__restrict__ dw)
{
    __shared__ float sm[32][NC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * NC + lane % NC;
    float s = 0.f;
    tc::grid_wait();
    if (c < cols) {
#pragma unroll 4
        for (int i = threadIdx.x / NC; i < nparts; i += 1024 / NC)
            s += part[i * cols + c];
    }
#pragma unroll
    for (int o = NC; o < 32; o *= 2)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane < NC)
        sm[warp][lane] = s;
    __syncthreads();
    if (threadIdx.x < NC && c < cols) {
        s = 0.f;
        for (int i = 0; i < 32; ++i)
            s += sm[i][lane];
        dw[c] = s;
    }
}

// warps and segments a row of `cols` columns takes: the first shape that
// holds it
#define NORM_SHAPES(X) X(1, 1) X(1, 2) X(4, 1) X(4, 2) X(8, 2) X(16, 2) X(32, 2) X(32, 4)
// of the backward kernel's eights: with its sums of dweight, 1024 threads of
// two segments lack registers (4096 x 16384 bf16: 114 us, 148 with X(32, 2))
#define NORM_SHAPES_BWD8(X) X(1, 1) X(1, 2) X(4, 1) X(4, 2) X(8, 2) X(16, 2) X(16, 4) X(32, 4)

// shared memory beyond the default is asked for once for each kernel and
// device (one bit of the mask)
template <typename F>
sg_status allow_smem(F *kernel, int bytes, std::atomic<uint64_t> &done)
{
    if (bytes <= 40 << 10)  // the default is 48 KB with the static part
        return SG_OK;
    int dev = 0;
    SG_TRY_CUDA(cudaGetDevice(&dev));
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        SG_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    return SG_OK;
}

// rows on their way: as many as leave room for the CTAs that fit by registers
template <typename T, int NA, int WARPS, int NV>
constexpr int ring_rows(int ctas)
{
    const int row = NA * NV * norm_threads(WARPS) * (int)sizeof(Pack8<T>);
    const int s = (216 << 10) / ctas / row;
    return s > 4 ? 4 : s < 1 ? 1 : s;
}

int64_t elem_size(int32_t dtype) { return dtype == SG_F32 ? 4 : 2; }

bool float_type(int32_t dtype) { return dtype == SG_BF16 || dtype == SG_F16 || dtype == SG_F32; }

// rows and columns of a row-wise operator, and every matrix's row stride
sg_status check_rows(const char *fn, int64_t nrows, int64_t cols, int32_t dtype)
{
    if (!float_type(dtype))
        NORM_FAIL(SG_ERR_INVALID, "%s: dtype %d is not SG_BF16, SG_F16 or SG_F32", fn, dtype);
    if (nrows < 0 || cols < 1)
        NORM_FAIL(SG_ERR_INVALID, "%s: need rows >= 0 and cols >= 1 (rows=%lld cols=%lld)", fn, (long long)nrows,
                  (long long)cols);
    if (nrows > INT32_MAX || cols > (1 << 30))
        NORM_FAIL(SG_ERR_UNSUPPORTED, "%s: rows=%lld or cols=%lld is above 2^31 - 1 or 2^30", fn, (long long)nrows,
                  (long long)cols);
    return SG_OK;
}

sg_status check_mat(const char *fn, const char *name, const void *p, int64_t ld, int64_t cols, int64_t elem)
{
    if (!p)
        return SG_OK;
    if (ld < cols)
        NORM_FAIL(SG_ERR_INVALID, "%s: the row stride of %s (%lld) is below its columns (%lld)", fn, name,
                  (long long)ld, (long long)cols);
    if (((uintptr_t)p) % elem != 0)
        NORM_FAIL(SG_ERR_INVALID, "%s: %s is not aligned to its elements", fn, name);
    return SG_OK;
}

// fp32 vectors
sg_status check_vec(const char *fn, const char *name, const void *p)
{
    if (((uintptr_t)p) % 4 != 0)
        NORM_FAIL(SG_ERR_INVALID, "%s: %s is not aligned to its elements", fn, name);
    return SG_OK;
}

}  // namespace
