// Activations kept in 8 bits (definitions in include/sg.h): rows to int8 with a
// scale for each group of 128 columns or for the row, and back.  Bound by
// memory: one read and one write of each.  32768 x 4096 bf16: to 8 bits 66 us (6.1
// TB/s), back 60 us (6.7 TB/s).
#include "norm.cuh"
#include "quant8.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kOut = 4;  // eights of a thread under way together

// i / n = (i magic) >> (32 + shift) for i < 2^31, with magic = ceil(2^(32 +
// shift) / n) and 2^shift < n <= 2^(shift + 1): the excess of magic, below n /
// 2^(32 + shift) of 1 / n, times i stays below 1 / n
struct Div {
    uint32_t n, magic, shift;

    explicit Div(uint32_t d) : n(d), magic(0), shift(0)
    {
        while ((2ull << shift) < d)
            ++shift;
        if (d > 1)
            magic = (uint32_t)(((1ull << (32 + shift)) + d - 1) / d);
    }
    __device__ __forceinline__ uint32_t of(uint32_t i) const
    {
        return n == 1 ? i : (uint32_t)(((uint64_t)i * magic) >> 32 >> shift);
    }
};

// Segments of 256 columns to 8 bits.  SPAN: a warp has kSpan of one row, next to
// each other; n, `spans` to a row, are numbered through all rows.  Else rows are
// short, and it has kOut of all rows' segments, a CTA's warps apart.  n is below
// 2^31 less those of a CTA.  The scales of a warp's groups are worked out together,
// a lane each, and a row's places once: 32768 x 4096 bf16 take 84 us with segments
// of any rows.
constexpr int kSpan = 4;

template <typename T, bool VEC, bool SPAN>
__global__ void __launch_bounds__(kThreads)
    k_pack_groups(const T *__restrict__ x, int64_t ldx, uint32_t n, const Div segs, int cols, int8_t *__restrict__ q,
                  int64_t ldq, float *__restrict__ scale)
{
    const int lane = threadIdx.x & 31, ng = (cols + kGroup - 1) / kGroup;
    if constexpr (SPAN) {
        const uint32_t i = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, r = segs.of(i);
        if (i >= n)
            return;
        const int c0 = (int)(i - r * segs.n) * kSpan * kSeg;
        const T *xr = x + r * ldx;
        int8_t *qr = q + r * ldq;
        float *sr = scale + (int64_t)r * ng;
        Pack8<T> p[kSpan];
#pragma unroll
        for (int k = 0; k < kSpan; ++k)
            p[k] = load8<T, VEC>(xr, c0 + k * kSeg, lane, cols);
        store_groups<T, VEC, kSpan>(
            p, lane, cols, [&](int) { return qr; }, [&](int) { return sr; }, [&](int k) { return c0 + k * kSeg; });
    } else {
        const uint32_t i0 = blockIdx.x * (kThreads / 32 * kOut) + threadIdx.x / 32;
        Pack8<T> p[kOut];
        uint32_t r[kOut];
        int c0[kOut];
#pragma unroll
        for (int k = 0; k < kOut; ++k) {
            const uint32_t i = i0 + k * (kThreads / 32);
            r[k] = segs.of(i);
            c0[k] = i < n ? (int)(i - r[k] * segs.n) * kSeg : cols;  // past the last: nothing of it is read or written
            p[k] = load8<T, VEC>(x + r[k] * ldx, c0[k], lane, cols);
        }
        store_groups<T, VEC, kOut>(
            p, lane, cols, [&](int k) { return q + r[k] * ldq; }, [&](int k) { return scale + (int64_t)r[k] * ng; },
            [&](int k) { return c0[k]; });
    }
}

// A row by WARPS warps (one warp: eight rows to a CTA), held in registers
// between its maximum and its use.
template <typename T, bool VEC, int WARPS, int NV>
__global__ void __launch_bounds__(norm_threads(WARPS))
    k_pack_rows(const T *__restrict__ x, int64_t ldx, int64_t nrows, int cols, int8_t *__restrict__ q, int64_t ldq,
                float *__restrict__ scale)
{
    __shared__ uint32_t sm[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int wr = WARPS == 1 ? 0 : warp;
    const int64_t r = WARPS == 1 ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
    if (r >= nrows)
        return;
    Pack8<T> p[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n)
        p[n] = load8<T, VEC>(x + r * ldx, (n * WARPS + wr) * kSeg, lane, cols);
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < NV; ++n)
        top = max(top, top8(p[n]));
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (WARPS > 1) {
        if (lane == 0)
            sm[warp] = top;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, sm[lane % WARPS]);
    }
    const Scale8 s = scale8_of(top);
    if (lane == 0 && wr == 0)
        scale[r] = s.scale;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        float2 v[4];
        unpack4(p[n], v);
        store8q<VEC>(q + r * ldq, (n * WARPS + wr) * kSeg, lane, cols, quant8(v, s.inv));
    }
}

// GROUPS: a scale for 128 columns, else for the row
template <typename T, bool VEC, bool GROUPS>
__global__ void __launch_bounds__(kThreads)
    k_unpack(const int8_t *__restrict__ q, int64_t ldq, const float *__restrict__ scale, uint32_t n, const Div segs,
             int cols, T *__restrict__ y, int64_t ldy)
{
    const int lane = threadIdx.x & 31, ng = (cols + kGroup - 1) / kGroup;
    const uint32_t i0 = blockIdx.x * (kThreads / 32 * kOut) + threadIdx.x / 32;
    uint2 w[kOut];
    float s[kOut], t[kOut];
#pragma unroll
    for (int k = 0; k < kOut; ++k) {
        const uint32_t i = i0 + k * (kThreads / 32);
        if (i < n) {
            const uint32_t r = segs.of(i);
            const int c0 = (int)(i - r * segs.n) * kSeg;
            w[k] = load8q<VEC>(q + r * ldq, c0, lane, cols);
            if (GROUPS) {
                // eights: the lane's group; else elements 0 to 3 and 4 to 7
                const float *at = scale + (int64_t)r * ng + c0 / kGroup;
                s[k] = VEC ? (c0 + lane * 8 < cols ? at[lane / 16] : 0.f) : at[0];
                t[k] = VEC ? s[k] : c0 + kGroup < cols ? at[1] : 0.f;
            } else {
                s[k] = t[k] = scale[r];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kOut; ++k) {
        const uint32_t i = i0 + k * (kThreads / 32);
        if (i >= n)
            return;
        const uint32_t r = segs.of(i);
        float2 v[4];
        unquant8(w[k], v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = mul2(v[j], both(j < 2 ? s[k] : t[k]));
        store8<T, VEC>(y + r * ldy, (int)(i - r * segs.n) * kSeg, lane, cols, pack4<T>(v));
    }
}

// rows of one launch of the kernels over segments
int64_t slab_of(int64_t segs) { return ((1ll << 31) - 1 - kThreads / 32 * kOut) / segs; }

unsigned grid_of(int64_t segments) { return (unsigned)ceil_div(segments, kThreads / 32 * kOut); }

template <typename T, bool VEC>
void run_pack(const void *x, int64_t ldx, int64_t nrows, int64_t cols, int32_t group, int8_t *q, int64_t ldq,
              float *scale, cudaStream_t st)
{
    const T *xs = static_cast<const T *>(x);
    if (group) {
        const int64_t segs = ceil_div(cols, kSeg), ng = ceil_div(cols, kGroup);
        // where at most a third of a row's spans would be empty
        const bool span = segs % kSpan == 0 || segs == 3 || segs >= 6;
        const int64_t per = span ? ceil_div(segs, kSpan) : segs, slab = slab_of(per);
        for (int64_t r0 = 0; r0 < nrows; r0 += slab) {
            const int64_t n = (nrows - r0 < slab ? nrows - r0 : slab) * per;
            const unsigned grid = span ? (unsigned)ceil_div(n, kThreads / 32) : grid_of(n);
            (span ? k_pack_groups<T, VEC, true> : k_pack_groups<T, VEC, false>)<<<grid, kThreads, 0, st>>>(
                xs + r0 * ldx, ldx, (uint32_t)n, Div((uint32_t)per), (int)cols, q + r0 * ldq, ldq, scale + r0 * ng);
        }
        return;
    }
#define X(W, N)                                                                                            \
    if (cols <= (int64_t)(W) * (N) * kSeg) {                                                               \
        k_pack_rows<T, VEC, W, N><<<(unsigned)((W) == 1 ? ceil_div(nrows, 8) : nrows), norm_threads(W), 0, st>>>( \
            xs, ldx, nrows, (int)cols, q, ldq, scale);                                                     \
        return;                                                                                            \
    }
    NORM_SHAPES(X)
#undef X
}

template <typename T, bool VEC>
void run_unpack(const int8_t *q, int64_t ldq, const float *scale, int64_t nrows, int64_t cols, int32_t group, void *y,
                int64_t ldy, cudaStream_t st)
{
    T *ys = static_cast<T *>(y);
    const int64_t segs = ceil_div(cols, kSeg), slab = slab_of(segs), ng = group ? ceil_div(cols, kGroup) : 1;
    for (int64_t r0 = 0; r0 < nrows; r0 += slab) {
        const int64_t n = (nrows - r0 < slab ? nrows - r0 : slab) * segs;
        if (group)
            k_unpack<T, VEC, true><<<grid_of(n), kThreads, 0, st>>>(q + r0 * ldq, ldq, scale + r0 * ng, (uint32_t)n,
                                                                    Div((uint32_t)segs), (int)cols, ys + r0 * ldy, ldy);
        else
            k_unpack<T, VEC, false><<<grid_of(n), kThreads, 0, st>>>(q + r0 * ldq, ldq, scale + r0 * ng, (uint32_t)n,
                                                                     Div((uint32_t)segs), (int)cols, ys + r0 * ldy, ldy);
    }
}

sg_status check_pack(const char *fn, const void *m, int64_t ldm, const char *name, int64_t nrows, int64_t cols,
                     int32_t dtype, int32_t group, const void *q, int64_t ldq, const float *scale)
{
    NORM_TRY(check_rows(fn, nrows, cols, dtype));
    if (group != 0 && group != kGroup)
        NORM_FAIL(SG_ERR_INVALID, "%s: group=%d is not 0 (the row) or %d", fn, group, kGroup);
    if (nrows && (!m || !q || !scale))
        NORM_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL", fn);
    NORM_TRY(check_mat(fn, name, m, ldm, cols, elem_size(dtype)));
    NORM_TRY(check_mat(fn, "q", q, ldq, cols, 1));
    return check_vec(fn, "scale", scale);
}

}  // namespace

extern "C" {

sg_status sg_pack8(const void *x, int64_t ldx, int64_t rows, int64_t cols, int32_t dtype, int32_t group, int8_t *q,
                   int64_t ldq, float *scale, void *stream)
{
    const char *fn = "sg_pack8";
    NvtxRange nvtx_(fn);
    NORM_TRY(check_pack(fn, x, ldx, "x", rows, cols, dtype, group, q, ldq, scale));
    if (!group && cols > kMaxCols)
        NORM_FAIL(SG_ERR_UNSUPPORTED, "%s: cols=%lld is above %lld with one scale for a row", fn, (long long)cols,
                  (long long)kMaxCols);
    if (rows == 0)
        return SG_OK;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = cols % 8 == 0 && vec_ok(x, ldx, elem_size(dtype)) && vec8_ok(q, ldq);
    if (dtype == SG_BF16)
        (vec ? run_pack<__nv_bfloat16, true> : run_pack<__nv_bfloat16, false>)(x, ldx, rows, cols, group, q, ldq, scale, st);
    else if (dtype == SG_F16)
        (vec ? run_pack<__half, true> : run_pack<__half, false>)(x, ldx, rows, cols, group, q, ldq, scale, st);
    else
        (vec ? run_pack<float, true> : run_pack<float, false>)(x, ldx, rows, cols, group, q, ldq, scale, st);
    SG_TRY_CUDA(cudaGetLastError());
    return SG_OK;
}

sg_status sg_unpack8(const int8_t *q, int64_t ldq, const float *scale, int64_t rows, int64_t cols, int32_t group,
                     void *y, int64_t ldy, int32_t dtype, void *stream)
{
    const char *fn = "sg_unpack8";
    NvtxRange nvtx_(fn);
    NORM_TRY(check_pack(fn, y, ldy, "y", rows, cols, dtype, group, q, ldq, scale));
    if (rows == 0)
        return SG_OK;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = cols % 8 == 0 && vec_ok(y, ldy, elem_size(dtype)) && vec8_ok(q, ldq);
    if (dtype == SG_BF16)
        (vec ? run_unpack<__nv_bfloat16, true> : run_unpack<__nv_bfloat16, false>)(q, ldq, scale, rows, cols, group, y, ldy, st);
    else if (dtype == SG_F16)
        (vec ? run_unpack<__half, true> : run_unpack<__half, false>)(q, ldq, scale, rows, cols, group, y, ldy, st);
    else
        (vec ? run_unpack<float, true> : run_unpack<float, false>)(q, ldq, scale, rows, cols, group, y, ldy, st);
    SG_TRY_CUDA(cudaGetLastError());
    return SG_OK;
}

}  // extern "C"
