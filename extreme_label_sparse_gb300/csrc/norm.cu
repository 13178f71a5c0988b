// Dropout and the residual's addition with RMS norm (definitions in
// include/sg.h).  All of them are bound by memory: each input is read once and
// each output written once.
#include <cmath>

#include <cuda_fp8.h>

#include "rows.cuh"

using namespace rows;

namespace {

#define NORM_FAIL(code, ...)       \
    do {                           \
        sg_set_error(__VA_ARGS__); \
        return code;               \
    } while (0)

constexpr int kDropThreads = 256;
constexpr int64_t kMaxCols = 32768;   // of the norm: a row lies in one CTA's registers
constexpr int kNormParts = 152 * 4;   // row groups that sum dweight before it is joined

// ---------------------------------------------------------------- dropout
// One warp per segment of 256 columns.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout(const T *x, int64_t ldx, int64_t nrows, int64_t cols, const Drop d, T *y, int64_t ldy)
{
    const int lane = threadIdx.x & 31;
    const int64_t segs = (cols + kSeg - 1) / kSeg;
    const int64_t step = (int64_t)gridDim.x * (kDropThreads / 32);
    for (int64_t i = (int64_t)blockIdx.x * (kDropThreads / 32) + threadIdx.x / 32; i < nrows * segs; i += step) {
        const int64_t r = i / segs, c0 = (i - r * segs) * kSeg;
        Pack8<T> p = load8<T, VEC>(x + r * ldx, c0, lane, cols);
        const uint32_t m = keep_lane<VEC>(d, c0, lane, (uint32_t)r);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p.v[j] = from_f<T>((m >> j) & 1u ? __fmul_rn(to_f(p.v[j]), d.scale) : 0.f);
        store8<T, VEC>(y + r * ldy, c0, lane, cols, p);
    }
}

// ---------------------------------------------------------------- norm
// Sum of a and maximum of b over the `warps` warps of a row group (all of the
// CTA where warps > 1).  Every thread gets both.
__device__ __forceinline__ void row_reduce(float &a, float &b, int warps, float2 *sm)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    if (warps == 1)
        return;
    __syncthreads();  // the last row's values have been read
    if ((threadIdx.x & 31) == 0)
        sm[threadIdx.x / 32] = make_float2(a, b);
    __syncthreads();
    a = 0.f;
    b = 0.f;
    for (int w = 0; w < warps; ++w) {
        a += sm[w].x;
        b = fmaxf(b, sm[w].y);
    }
}

struct NormFwd {
    const void *x, *res, *w;
    void *u, *y;
    uint8_t *y8;
    float *rstd, *scale8;
    int64_t ldx, ldr, ldu, ldy, ld8, nrows, cols;
    float eps;
    Drop d;
};

// A row by WARPS warps (one warp: eight rows to a CTA), NV segments to a warp.
template <typename T, bool VEC, int WARPS, int NV>
__global__ void __launch_bounds__(WARPS == 1 ? 256 : WARPS * 32) k_norm_fwd(const NormFwd a)
{
    __shared__ float2 sm[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int wr = WARPS == 1 ? 0 : warp;
    const int64_t r = WARPS == 1 ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
    if (r >= a.nrows)  // whole warps, and never a part of a CTA that meets in row_reduce
        return;
    float v[NV][8];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int64_t c0 = (int64_t)(n * WARPS + wr) * kSeg;
        Pack8<T> p = load8<T, VEC>(static_cast<const T *>(a.x) + r * a.ldx, c0, lane, a.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[n][j] = to_f(p.v[j]);
        if (a.d.drop) {
            const uint32_t m = keep_lane<VEC>(a.d, c0, lane, (uint32_t)r);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[n][j] = (m >> j) & 1u ? __fmul_rn(v[n][j], a.d.scale) : 0.f;
        }
        if (a.res) {
            const Pack8<T> q = load8<T, VEC>(static_cast<const T *>(a.res) + r * a.ldr, c0, lane, a.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[n][j] = __fadd_rn(v[n][j], to_f(q.v[j]));
        }
        // the norm is taken of the sum as it is stored, so that the backward
        // pass sees the same row
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p.v[j] = from_f<T>(v[n][j]);
        if (a.u)
            store8<T, VEC>(static_cast<T *>(a.u) + r * a.ldu, c0, lane, a.cols, p);
        const Pack8<T> w = load8<T, VEC>(static_cast<const T *>(a.w), c0, lane, a.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[n][j] = to_f(p.v[j]);
            ss = fmaf(v[n][j], v[n][j], ss);
            top = fmaxf(top, fabsf(v[n][j] * to_f(w.v[j])));
        }
    }
    row_reduce(ss, top, WARPS, sm);
    const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
    // max |y| without a second reduction: rstd max |u w|
    top *= rstd;
    const float to8 = top == 0.f ? 0.f : 448.0f / top;
    if (lane == 0 && wr == 0) {
        if (a.rstd)
            a.rstd[r] = rstd;
        if (a.y8)
            a.scale8[r] = top / 448.0f;
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int64_t c0 = (int64_t)(n * WARPS + wr) * kSeg;
        const Pack8<T> w = load8<T, VEC>(static_cast<const T *>(a.w), c0, lane, a.cols);
        Pack8<T> p;
        Pack8<uint8_t> q;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = (v[n][j] * rstd) * to_f(w.v[j]);
            p.v[j] = from_f<T>(y);
            q.v[j] = __nv_cvt_float_to_fp8(y * to8, __NV_SATFINITE, __NV_E4M3);
        }
        if (a.y)
            store8<T, VEC>(static_cast<T *>(a.y) + r * a.ldy, c0, lane, a.cols, p);
        if (a.y8) {
            uint8_t *row = a.y8 + r * a.ld8;
            if constexpr (VEC) {
                if (c0 + lane * 8 < a.cols)
                    *reinterpret_cast<uint2 *>(row + c0 + lane * 8) = *reinterpret_cast<const uint2 *>(&q);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col_of<VEC>(c0, lane, j) < a.cols)
                        row[col_of<VEC>(c0, lane, j)] = q.v[j];
            }
        }
    }
}

struct NormBwd {
    const void *dy, *u, *w, *du_in;
    const float *rstd;
    void *du, *dx;
    float *part;  // [row groups][cols], or NULL: no dweight
    int64_t lddy, ldu, ldi, ldo, lddx, nrows, cols;
    Drop d;
};

// Row groups of WARPS warps step over the rows; a thread keeps the sum of its
// columns of dweight in registers until its last row.
template <typename T, bool VEC, int WARPS, int NV>
__global__ void __launch_bounds__(WARPS == 1 ? 256 : WARPS * 32) k_norm_bwd(const NormBwd a)
{
    __shared__ float2 sm[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int wr = WARPS == 1 ? 0 : warp;
    const int64_t groups = WARPS == 1 ? (int64_t)gridDim.x * 8 : (int64_t)gridDim.x;
    const int64_t g = WARPS == 1 ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
    float dw[NV][8] = {};
    for (int64_t r = g; r < a.nrows; r += groups) {
        Pack8<T> dy[NV], u[NV];
        const float rstd = a.rstd[r];
        float dot = 0.f, none = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int64_t c0 = (int64_t)(n * WARPS + wr) * kSeg;
            dy[n] = load8<T, VEC>(static_cast<const T *>(a.dy) + r * a.lddy, c0, lane, a.cols);
            u[n] = load8<T, VEC>(static_cast<const T *>(a.u) + r * a.ldu, c0, lane, a.cols);
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int64_t c0 = (int64_t)(n * WARPS + wr) * kSeg;
            const Pack8<T> w = load8<T, VEC>(static_cast<const T *>(a.w), c0, lane, a.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = to_f(dy[n].v[j]) * (to_f(u[n].v[j]) * rstd);
                dw[n][j] += t;
                dot = fmaf(t, to_f(w.v[j]), dot);
            }
        }
        row_reduce(dot, none, WARPS, sm);
        const float mean = dot / (float)a.cols;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int64_t c0 = (int64_t)(n * WARPS + wr) * kSeg;
            const Pack8<T> w = load8<T, VEC>(static_cast<const T *>(a.w), c0, lane, a.cols);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = rstd * (to_f(dy[n].v[j]) * to_f(w.v[j]) - (to_f(u[n].v[j]) * rstd) * mean);
            if (a.du_in) {
                const Pack8<T> q = load8<T, VEC>(static_cast<const T *>(a.du_in) + r * a.ldi, c0, lane, a.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += to_f(q.v[j]);
            }
            Pack8<T> p;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                p.v[j] = from_f<T>(v[j]);
            store8<T, VEC>(static_cast<T *>(a.du) + r * a.ldo, c0, lane, a.cols, p);
            if (a.dx) {
                if (a.d.drop) {
                    const uint32_t m = keep_lane<VEC>(a.d, c0, lane, (uint32_t)r);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        p.v[j] = from_f<T>((m >> j) & 1u ? v[j] * a.d.scale : 0.f);
                }
                store8<T, VEC>(static_cast<T *>(a.dx) + r * a.lddx, c0, lane, a.cols, p);
            }
        }
    }
    if (a.part) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t c = col_of<VEC>((int64_t)(n * WARPS + wr) * kSeg, lane, j);
                if (c < a.cols)
                    a.part[g * a.cols + c] = dw[n][j];
            }
    }
}

// dweight[c] = the sum of its parts, in a fixed order
__global__ void __launch_bounds__(1024) k_norm_dw(const float *__restrict__ part, int nparts, int64_t cols,
                                                  float *__restrict__ dw)
{
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols)
        for (int i = warp; i < nparts; i += 32)
            s += part[i * cols + c];
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
        s = 0.f;
        for (int i = 0; i < 32; ++i)
            s += sm[i][lane];
        dw[c] = s;
    }
}

// warps and segments a row of `cols` columns takes: the first shape that
// holds it
#define NORM_SHAPES(X) X(1, 1) X(1, 2) X(1, 4) X(4, 2) X(8, 2) X(16, 2) X(16, 4) X(32, 4)

template <typename T, bool VEC>
void launch_fwd(const NormFwd &a, cudaStream_t st)
{
#define X(W, N)                                                                                  \
    if (a.cols <= (int64_t)(W) * (N) * kSeg) {                                                   \
        const int64_t grid = (W) == 1 ? ceil_div(a.nrows, 8) : a.nrows;                          \
        k_norm_fwd<T, VEC, W, N><<<(unsigned)grid, (W) == 1 ? 256 : (W) * 32, 0, st>>>(a);       \
        return;                                                                                  \
    }
    NORM_SHAPES(X)
#undef X
}

// CTAs of the backward kernel, and the row groups they make
int64_t bwd_groups(int64_t nrows, int64_t cols, int64_t *grid)
{
    const bool one = cols <= 4 * kSeg;  // one warp to a row
    const int64_t most = one ? kNormParts / 8 * 2 : kNormParts;
    const int64_t need = one ? ceil_div(nrows, 8) : nrows;
    *grid = need < most ? need : most;
    return one ? *grid * 8 : *grid;
}

template <typename T, bool VEC>
void launch_bwd(const NormBwd &a, int64_t grid, cudaStream_t st)
{
#define X(W, N)                                                                                  \
    if (a.cols <= (int64_t)(W) * (N) * kSeg) {                                                   \
        k_norm_bwd<T, VEC, W, N><<<(unsigned)grid, (W) == 1 ? 256 : (W) * 32, 0, st>>>(a);       \
        return;                                                                                  \
    }
    NORM_SHAPES(X)
#undef X
}

template <typename T>
void launch_dropout(bool vec, const void *x, int64_t ldx, int64_t nrows, int64_t cols, const Drop &d, void *y,
                    int64_t ldy, cudaStream_t st)
{
    const int64_t warps = nrows * ceil_div(cols, kSeg);
    int64_t grid = ceil_div(warps, kDropThreads / 32);
    if (grid > (1 << 20))
        grid = 1 << 20;
    const T *xs = static_cast<const T *>(x);
    T *ys = static_cast<T *>(y);
    if (vec)
        k_dropout<T, true><<<(unsigned)grid, kDropThreads, 0, st>>>(xs, ldx, nrows, cols, d, ys, ldy);
    else
        k_dropout<T, false><<<(unsigned)grid, kDropThreads, 0, st>>>(xs, ldx, nrows, cols, d, ys, ldy);
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
    if (nrows > INT32_MAX || cols > INT32_MAX)
        NORM_FAIL(SG_ERR_UNSUPPORTED, "%s: rows and cols must be below 2^31 (rows=%lld cols=%lld)", fn,
                  (long long)nrows, (long long)cols);
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

#define NORM_TRY(expr)          \
    do {                        \
        sg_status rc_ = (expr); \
        if (rc_ != SG_OK)       \
            return rc_;         \
    } while (0)

}  // namespace

extern "C" {

sg_status sg_dropout(const void *x, int64_t ldx, int64_t rows, int64_t cols, int32_t dtype, double p, uint64_t seed,
                     uint64_t offset, void *y, int64_t ldy, void *stream)
{
    const char *fn = "sg_dropout";
    NvtxRange nvtx_(fn);
    NORM_TRY(check_rows(fn, rows, cols, dtype));
    if (rows && (!x || !y))
        NORM_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL", fn);
    const int64_t es = elem_size(dtype);
    NORM_TRY(check_mat(fn, "x", x, ldx, cols, es));
    NORM_TRY(check_mat(fn, "y", y, ldy, cols, es));
    Drop d;
    if (!make_drop(p, seed, offset, &d))
        NORM_FAIL(SG_ERR_INVALID, "%s: p=%g is not a probability", fn, p);
    if (rows == 0)
        return SG_OK;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = cols % 8 == 0 && vec_ok(x, ldx, es) && vec_ok(y, ldy, es);
    if (dtype == SG_BF16)
        launch_dropout<__nv_bfloat16>(vec, x, ldx, rows, cols, d, y, ldy, st);
    else if (dtype == SG_F16)
        launch_dropout<__half>(vec, x, ldx, rows, cols, d, y, ldy, st);
    else
        launch_dropout<float>(vec, x, ldx, rows, cols, d, y, ldy, st);
    SG_TRY_CUDA(cudaGetLastError());
    return SG_OK;
}

sg_status sg_add_rmsnorm_fwd(const void *x, int64_t ldx, const void *residual, int64_t ldr, int64_t rows,
                             int64_t cols, int32_t dtype, const void *weight, double eps, double drop_p,
                             uint64_t seed, uint64_t offset, void *u, int64_t ldu, float *rstd, void *y, int64_t ldy,
                             uint8_t *y8, int64_t ldy8, float *y8_scale, void *stream)
{
    const char *fn = "sg_add_rmsnorm_fwd";
    NvtxRange nvtx_(fn);
    NORM_TRY(check_rows(fn, rows, cols, dtype));
    if (cols > kMaxCols)
        NORM_FAIL(SG_ERR_UNSUPPORTED, "%s: cols=%lld is above %lld", fn, (long long)cols, (long long)kMaxCols);
    if (!weight || (rows && (!x || (!y && !y8) || (y8 && !y8_scale))))
        NORM_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL (x, weight, y or y8, y8's scales)", fn);
    if (!(eps >= 0.0) || !std::isfinite(eps))
        NORM_FAIL(SG_ERR_INVALID, "%s: eps=%g is not a finite number >= 0", fn, eps);
    const int64_t es = elem_size(dtype);
    NORM_TRY(check_mat(fn, "x", x, ldx, cols, es));
    NORM_TRY(check_mat(fn, "residual", residual, ldr, cols, es));
    NORM_TRY(check_mat(fn, "weight", weight, cols, cols, es));
    NORM_TRY(check_mat(fn, "u", u, ldu, cols, es));
    NORM_TRY(check_mat(fn, "y", y, ldy, cols, es));
    NORM_TRY(check_mat(fn, "y8", y8, ldy8, cols, 1));
    NormFwd a;
    if (!make_drop(drop_p, seed, offset, &a.d))
        NORM_FAIL(SG_ERR_INVALID, "%s: drop_p=%g is not a probability", fn, drop_p);
    if (rows == 0)
        return SG_OK;
    a.x = x, a.res = residual, a.w = weight, a.u = u, a.y = y, a.y8 = y8, a.rstd = rstd, a.scale8 = y8_scale;
    a.ldx = ldx, a.ldr = ldr, a.ldu = ldu, a.ldy = ldy, a.ld8 = ldy8, a.nrows = rows, a.cols = cols;
    a.eps = (float)eps;
    cudaStream_t st = (cudaStream_t)stream;
    // 8-bit rows are written in pieces of 8 bytes: half the 16 that vec_ok asks
    const bool vec = cols % 8 == 0 && vec_ok(x, ldx, es) && vec_ok(residual, ldr, es) && vec_ok(weight, cols, es) &&
                     vec_ok(u, ldu, es) && vec_ok(y, ldy, es) && (!y8 || (((uintptr_t)y8) % 8 == 0 && ldy8 % 8 == 0));
    if (dtype == SG_BF16)
        vec ? launch_fwd<__nv_bfloat16, true>(a, st) : launch_fwd<__nv_bfloat16, false>(a, st);
    else if (dtype == SG_F16)
        vec ? launch_fwd<__half, true>(a, st) : launch_fwd<__half, false>(a, st);
    else
        vec ? launch_fwd<float, true>(a, st) : launch_fwd<float, false>(a, st);
    SG_TRY_CUDA(cudaGetLastError());
    return SG_OK;
}

sg_status sg_add_rmsnorm_bwd_work(int64_t rows, int64_t cols, int64_t *bytes)
{
    const char *fn = "sg_add_rmsnorm_bwd_work";
    if (!bytes)
        NORM_FAIL(SG_ERR_INVALID, "%s: bytes is NULL", fn);
    NORM_TRY(check_rows(fn, rows, cols, SG_F32));
    if (cols > kMaxCols)
        NORM_FAIL(SG_ERR_UNSUPPORTED, "%s: cols=%lld is above %lld", fn, (long long)cols, (long long)kMaxCols);
    int64_t grid;
    *bytes = bwd_groups(rows, cols, &grid) * cols * 4;
    return SG_OK;
}

sg_status sg_add_rmsnorm_bwd(const void *dy, int64_t lddy, const void *u, int64_t ldu, const void *du_in,
                             int64_t lddu_in, int64_t rows, int64_t cols, int32_t dtype, const void *weight,
                             const float *rstd, double drop_p, uint64_t seed, uint64_t offset, void *du, int64_t lddu,
                             void *dx, int64_t lddx, float *dweight, void *work, int64_t work_bytes, void *stream)
{
    const char *fn = "sg_add_rmsnorm_bwd";
    NvtxRange nvtx_(fn);
    NORM_TRY(check_rows(fn, rows, cols, dtype));
    if (cols > kMaxCols)
        NORM_FAIL(SG_ERR_UNSUPPORTED, "%s: cols=%lld is above %lld", fn, (long long)cols, (long long)kMaxCols);
    if (!weight || (rows && (!dy || !u || !rstd || !du)))
        NORM_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL (dy, u, weight, rstd, du)", fn);
    const int64_t es = elem_size(dtype);
    NORM_TRY(check_mat(fn, "dy", dy, lddy, cols, es));
    NORM_TRY(check_mat(fn, "u", u, ldu, cols, es));
    NORM_TRY(check_mat(fn, "du_in", du_in, lddu_in, cols, es));
    NORM_TRY(check_mat(fn, "weight", weight, cols, cols, es));
    NORM_TRY(check_mat(fn, "du", du, lddu, cols, es));
    NORM_TRY(check_mat(fn, "dx", dx, lddx, cols, es));
    NormBwd a;
    if (!make_drop(drop_p, seed, offset, &a.d))
        NORM_FAIL(SG_ERR_INVALID, "%s: drop_p=%g is not a probability", fn, drop_p);
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        if (dweight)
            SG_TRY_CUDA(cudaMemsetAsync(dweight, 0, (size_t)cols * 4, st));
        return SG_OK;
    }
    int64_t grid;
    const int64_t groups = bwd_groups(rows, cols, &grid);
    if (dweight && (!work || work_bytes < groups * cols * 4 || ((uintptr_t)work) % 4 != 0))
        NORM_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_add_rmsnorm_bwd_work), aligned to 4", fn,
                  (long long)(groups * cols * 4));
    a.dy = dy, a.u = u, a.w = weight, a.du_in = du_in, a.rstd = rstd, a.du = du, a.dx = dx;
    a.part = dweight ? static_cast<float *>(work) : nullptr;
    a.lddy = lddy, a.ldu = ldu, a.ldi = lddu_in, a.ldo = lddu, a.lddx = lddx, a.nrows = rows, a.cols = cols;
    const bool vec = cols % 8 == 0 && vec_ok(dy, lddy, es) && vec_ok(u, ldu, es) && vec_ok(du_in, lddu_in, es) &&
                     vec_ok(weight, cols, es) && vec_ok(du, lddu, es) && vec_ok(dx, lddx, es);
    if (dtype == SG_BF16)
        vec ? launch_bwd<__nv_bfloat16, true>(a, grid, st) : launch_bwd<__nv_bfloat16, false>(a, grid, st);
    else if (dtype == SG_F16)
        vec ? launch_bwd<__half, true>(a, grid, st) : launch_bwd<__half, false>(a, grid, st);
    else
        vec ? launch_bwd<float, true>(a, grid, st) : launch_bwd<float, false>(a, grid, st);
    SG_TRY_CUDA(cudaGetLastError());
    if (dweight) {
        k_norm_dw<<<(unsigned)ceil_div(cols, 32), 1024, 0, st>>>(a.part, (int)groups, cols, dweight);
        SG_TRY_CUDA(cudaGetLastError());
    }
    return SG_OK;
}

}  // extern "C"
