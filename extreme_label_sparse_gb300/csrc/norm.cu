// Dropout and the residual's addition with RMS norm (definitions in
// include/sg.h).  All of them are bound by memory: each input is read once and
// each output written once, but for the backward kernel's rows that are not
// whole, aligned eights, of which dy and u are read twice (mostly from the
// caches the second time).
#include <atomic>
#include <cmath>

#include <cuda_fp8.h>

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

constexpr int kDropThreads = 256, kDropCtas = 6;
constexpr int drop_u(int size) { return size == 4 ? 2 : 4; }  // blocks of a thread: 64 bytes
constexpr int64_t kMaxCols = 32768;   // of the norm: a row lies in one CTA's registers
constexpr int kSMs = 152;

// ---------------------------------------------------------------- dropout
// One warp for a segment of 256 columns: any alignment and width.  segs
// (segments of a row) times rows is below 2^31.  Bound by the accesses of one
// element to a lane: 65536 x 1001 bf16 take 76 us (3.5 TB/s), half the rate of
// rows of whole eights.
template <typename T>
__global__ void __launch_bounds__(kDropThreads, kDropCtas)
    k_dropout_any(const T *x, int64_t ldx, uint32_t nseg, uint32_t segs, int cols, uint32_t row0, const Drop d, T *y,
                  int64_t ldy)
{
    const int lane = threadIdx.x & 31;
    const uint32_t i = blockIdx.x * (kDropThreads / 32) + threadIdx.x / 32;
    if (i >= nseg)
        return;
    const uint32_t r = i / segs;
    const int c0 = (int)(i - r * segs) * kSeg;
    Pack8<T> p = load8<T, false>(x + r * ldx, c0, lane, cols);
    if (d.drop) {
        const Keep<false> k(d, c0, lane, row0 + r);
        float v[8];
        unpack8(p, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = k.at(j) ? __fmul_rn(v[j], d.scale) : 0.f;
        p = pack8<T>(v);
    }
    store8<T, false>(y + r * ldy, c0, lane, cols, p);
}

// Rows of whole, aligned eights: the blocks of all rows are numbered through,
// and a thread takes U of them, kDropThreads apart, whose loads it issues
// together.  n (blocks) is below 2^31; row = i / blks by a multiplication.
// DENSE: no gaps between rows.  The copy alone would take as long as long as
// loads stay ahead of the rounds (about 140 instructions for eight elements):
// four at once and 1536 threads to an SM reach it, 79 us for 32768 x 4096 bf16
// (6.8 TB/s); two at once take 86, a loop with the next load ahead 102.
template <typename T, bool DENSE>
__global__ void __launch_bounds__(kDropThreads, kDropCtas)
    k_dropout(const T *x, int64_t ldx, uint32_t n, uint32_t blks, uint32_t magic, uint32_t shift, uint32_t row0,
              const Drop d, T *y, int64_t ldy)
{
    constexpr int U = drop_u(sizeof(T));
    const uint32_t i0 = blockIdx.x * (kDropThreads * U) + threadIdx.x;
    auto row_of = [&](uint32_t i) { return blks == 1 ? i : (uint32_t)(((uint64_t)i * magic) >> 32 >> shift); };
    auto at = [&](uint32_t i, int64_t ld) {
        if (DENSE)
            return (int64_t)i * 8;
        const uint32_t r = row_of(i);
        return r * ld + (i - r * blks) * 8;
    };
    Pack8<T> p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + u * kDropThreads;
        if (i < n)
            p[u] = load_pack(x + at(i, ldx));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + u * kDropThreads;
        if (i >= n)
            return;
        if (d.drop) {
            const uint32_t r = row_of(i);
            const Keep<true> k(d, (int)(i - r * blks) * 8, 0, row0 + r);
            float v[8];
            unpack8(p[u], v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = k.at(j) ? __fmul_rn(v[j], d.scale) : 0.f;
            p[u] = pack8<T>(v);
        }
        store_pack(y + at(i, ldy), p[u]);
    }
}

// ---------------------------------------------------------------- norm
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
// The forward kernel takes 512 with fp32 and with three segments to a warp,
// which lack registers otherwise (65536 x 768 bf16 to 8 bits with dropout: 68
// us, 81 with 1024; 16384 x 4096 to 8 bits, two segments: 79 us, 75 with 1024).
constexpr int fwd_ctas(int warps, int nv, int size) { return norm_ctas(warps, size == 4 || nv == 3); }
// The backward kernel's eights take 512 in all types: its sums of dweight spill
// otherwise (16384 x 4096 bf16 with dropout: 107 us, 124 with 1024).  Single
// elements, with no ring of rows, want the warps even though their 64 registers
// spill at most widths (32768 x 1001 with dropout: 97 us, 140 with 512).
constexpr int bwd_ctas(bool vec, int warps, int size) { return norm_ctas(warps, size == 4 || vec); }

struct NormFwd {
    const void *x, *res, *w;
    void *u, *y;
    uint8_t *y8;
    float *rstd, *scale8;
    int64_t ldx, ldr, ldu, ldy, ld8, nrows;
    int cols;
    float eps;
    Drop d;
};

// A row by WARPS warps (one warp: eight rows to a CTA), NV segments to a warp.
// Row groups step over the rows.  The row stays in registers between the sum
// of its squares and its use, so each input is read once; the next rows are on
// their way to shared memory meanwhile, since a CTA that waits for its row's
// sum would otherwise have nothing in flight (16384 x 4096 bf16, sum and 8-bit
// outputs: 100 us with loads into registers, now 74.5 us, 6.3 TB/s; 2.4 us for
// 128 x 768).  No barrier but the sum's own; wide rows take several
// warps, so that a thread has at most two segments in registers.
template <typename T, bool VEC, int WARPS, int NV, int S>
__global__ void __launch_bounds__(norm_threads(WARPS), fwd_ctas(WARPS, NV, sizeof(T))) k_norm_fwd(const NormFwd a)
{
    __shared__ RowSums sm;
    extern __shared__ uint4 dyn[];
    const Ring8<T, 2, NV, S, norm_threads(WARPS)> ring(dyn);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int wr = WARPS == 1 ? 0 : warp;
    const int64_t groups = WARPS == 1 ? (int64_t)gridDim.x * 8 : (int64_t)gridDim.x;
    const int64_t g = WARPS == 1 ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
    const T *ax = static_cast<const T *>(a.x), *ar = static_cast<const T *>(a.res);
    auto fetch = [&](int64_t r, int slot) {
        if constexpr (VEC) {
            if (r < a.nrows) {
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int c = (n * WARPS + wr) * kSeg + lane * 8;
                    if (c < a.cols) {
                        ring.copy(slot, 0, n, ax + r * a.ldx + c);
                        if (ar)
                            ring.copy(slot, 1, n, ar + r * a.ldr + c);
                    }
                }
            }
            copies_commit();
        }
    };
#pragma unroll
    for (int i = 0; i < S; ++i)
        fetch(g + i * groups, i);
    Pack8<T> w[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n)
        w[n] = load8<T, VEC>(static_cast<const T *>(a.w), (n * WARPS + wr) * kSeg, lane, a.cols);
    int turn = 0, slot = 0;
    for (int64_t r = g; r < a.nrows; r += groups, ++turn) {
        Pack8<T> u[NV];
        float ss = 0.f, top = 0.f;
        if constexpr (VEC)
            copies_wait<S - 1>();
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c0 = (n * WARPS + wr) * kSeg;
            if (VEC && c0 + lane * 8 >= a.cols)
                break;  // and neither has a later segment columns of this thread
            Pack8<T> p;
            if constexpr (VEC)
                p = ring.get(slot, 0, n);
            else
                p = load8<T, VEC>(ax + r * a.ldx, c0, lane, a.cols);
            float v[8];
            unpack8(p, v);
            if (a.d.drop) {
                const Keep<VEC> k(a.d, c0, lane, (uint32_t)r);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = k.at(j) ? __fmul_rn(v[j], a.d.scale) : 0.f;
            }
            if (ar) {
                if constexpr (VEC)
                    p = ring.get(slot, 1, n);
                else
                    p = load8<T, VEC>(ar + r * a.ldr, c0, lane, a.cols);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = __fadd_rn(v[j], to_f(p.v[j]));
            }
            // the norm is taken of the sum as it is stored, so that the
            // backward pass sees the same row
            u[n] = pack8<T>(v);
            unpack8(u[n], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(v[j], v[j], ss);
                top = fmaxf(top, fabsf(v[j] * to_f(w[n].v[j])));
            }
            if (a.u)
                store8<T, VEC>(static_cast<T *>(a.u) + r * a.ldu, c0, lane, a.cols, u[n]);
        }
        fetch(r + S * groups, slot);
        slot = slot + 1 == S ? 0 : slot + 1;
        row_reduce<WARPS, true>(ss, top, sm, turn);
        const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        // max |y| without a second reduction: rstd max |u w|
        top *= rstd;
        // scales of at least 2^-126: below, 1 / scale would not be an fp32 number
        const float to8 = top == 0.f ? 0.f : top < 448.0f * 0x1p-126f ? 0x1p126f : 448.0f / top;
        if (lane == 0 && wr == 0) {
            if (a.rstd)
                a.rstd[r] = rstd;
            if (a.y8)
                a.scale8[r] = top > 0.f && top < 448.0f * 0x1p-126f ? 0x1p-126f : top / 448.0f;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c0 = (n * WARPS + wr) * kSeg;
            if (VEC && c0 + lane * 8 >= a.cols)
                break;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = (to_f(u[n].v[j]) * rstd) * to_f(w[n].v[j]);
            if (a.y) {
                store8<T, VEC>(static_cast<T *>(a.y) + r * a.ldy, c0, lane, a.cols, pack8<T>(y));
            }
            if (a.y8) {
                uint8_t *row = a.y8 + r * a.ld8;
                uint16_t q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    q[j] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * j] * to8, y[2 * j + 1] * to8), __NV_SATFINITE,
                                                    __NV_E4M3);
                if constexpr (VEC) {
                    *reinterpret_cast<uint2 *>(row + c0 + lane * 8) =
                        make_uint2(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col_of<VEC>(c0, lane, j) < a.cols)
                            row[col_of<VEC>(c0, lane, j)] = (uint8_t)(q[j / 2] >> (8 * (j & 1)));
                }
            }
        }
    }
}

struct NormBwd {
    const void *dy, *u, *w, *du_in;
    const float *rstd;
    void *du, *dx;
    float *part;  // [row groups][cols], or NULL: no dweight
    int64_t lddy, ldu, ldi, ldo, lddx, nrows;
    int cols;
    Drop d;
};

// Row groups of WARPS warps step over the rows; a thread keeps the sum of its
// columns of dweight in registers until its last row, and the groups' sums are
// joined by k_norm_dw.  Both uses of dy and u are served from shared memory, so
// memory is read once: 16384 x 4096 bf16 with du_in and dropout, 671 MB, 107
// us (6.3 TB/s; 189 us with loads into registers, 139 with rstd read in its own
// turn).
template <typename T, bool VEC, int WARPS, int NV, int S>
__global__ void __launch_bounds__(norm_threads(WARPS), bwd_ctas(VEC, WARPS, sizeof(T))) k_norm_bwd(const NormBwd a)
{
    __shared__ RowSums sm;
    extern __shared__ uint4 dyn[];
    const Ring8<T, 3, NV, S, norm_threads(WARPS)> ring(dyn);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int wr = WARPS == 1 ? 0 : warp;
    const int64_t groups = WARPS == 1 ? (int64_t)gridDim.x * 8 : (int64_t)gridDim.x;
    const int64_t g = WARPS == 1 ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
    tc::grid_go();
    const T *ady = static_cast<const T *>(a.dy), *au = static_cast<const T *>(a.u);
    const T *ai = static_cast<const T *>(a.du_in);
    auto fetch = [&](int64_t r, int slot) {
        if constexpr (VEC) {
            if (r < a.nrows) {
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int c = (n * WARPS + wr) * kSeg + lane * 8;
                    if (c < a.cols) {
                        ring.copy(slot, 0, n, ady + r * a.lddy + c);
                        ring.copy(slot, 1, n, au + r * a.ldu + c);
                        if (ai)
                            ring.copy(slot, 2, n, ai + r * a.ldi + c);
                    }
                }
            }
            copies_commit();
        }
    };
#pragma unroll
    for (int i = 0; i < S; ++i)
        fetch(g + i * groups, i);
    Pack8<T> w[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n)
        w[n] = load8<T, VEC>(static_cast<const T *>(a.w), (n * WARPS + wr) * kSeg, lane, a.cols);
    float dw[NV][8] = {};
    int turn = 0, slot = 0;
    // rstd is read ahead, or each row would begin with a wait for it: one row, or
    // with four segments, which have few rows to a CTA, 32 rows at a time by the
    // lanes (16384 x 4096 bf16: 107 us, 110 by the lanes; 4096 x 16384: 139, 114)
    constexpr bool kLanes = NV == 4;
    float next = kLanes || g >= a.nrows ? 0.f : a.rstd[g];
    for (int64_t r = g; r < a.nrows; r += groups, ++turn) {
        float rstd;
        if constexpr (kLanes) {
            if ((turn & 31) == 0)
                next = r + lane * groups < a.nrows ? a.rstd[r + lane * groups] : 0.f;
            rstd = __shfl_sync(0xffffffffu, next, turn & 31);
        } else {
            rstd = next;
            if (r + groups < a.nrows)
                next = a.rstd[r + groups];
        }
        float dot = 0.f, none = 0.f;
        if constexpr (VEC)
            copies_wait<S - 1>();
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c0 = (n * WARPS + wr) * kSeg;
            if (VEC && c0 + lane * 8 >= a.cols)
                break;  // and neither has a later segment columns of this thread
            Pack8<T> dy, u;
            if constexpr (VEC) {
                dy = ring.get(slot, 0, n);
                u = ring.get(slot, 1, n);
            } else {
                dy = load8<T, VEC>(ady + r * a.lddy, c0, lane, a.cols);
                u = load8<T, VEC>(au + r * a.ldu, c0, lane, a.cols);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = to_f(dy.v[j]) * to_f(u.v[j]);
                dw[n][j] = fmaf(t, rstd, dw[n][j]);
                dot = fmaf(t, to_f(w[n].v[j]), dot);
            }
        }
        row_reduce<WARPS, false>(dot, none, sm, turn);
        // du = rstd (dy w - n mean(dy w n)): (rstd w) dy - back n with n = u
        // rstd, back = rstd mean(dy w n).  Neither a square of u nor one of rstd
        // is a part of it without the other, which leaves rows of values from
        // 1e-36 to 1e34 within the range of fp32.
        const float back = dot / (float)a.cols * rstd * rstd;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c0 = (n * WARPS + wr) * kSeg;
            if (VEC && c0 + lane * 8 >= a.cols)
                break;
            // once more from shared memory (or, without VEC, from the caches)
            Pack8<T> dy, u;
            if constexpr (VEC) {
                dy = ring.get(slot, 0, n);
                u = ring.get(slot, 1, n);
            } else {
                dy = load8<T, VEC>(ady + r * a.lddy, c0, lane, a.cols);
                u = load8<T, VEC>(au + r * a.ldu, c0, lane, a.cols);
            }
            float v[8];
            if (ai) {
                Pack8<T> in;
                if constexpr (VEC)
                    in = ring.get(slot, 2, n);
                else
                    in = load8<T, VEC>(ai + r * a.ldi, c0, lane, a.cols);
                unpack8(in, v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = fmaf(to_f(w[n].v[j]) * rstd, to_f(dy.v[j]), fmaf(-back, to_f(u.v[j]) * rstd, v[j]));
            store8<T, VEC>(static_cast<T *>(a.du) + r * a.ldo, c0, lane, a.cols, pack8<T>(v));
            if (a.dx) {
                if (a.d.drop) {
                    const Keep<VEC> k(a.d, c0, lane, (uint32_t)r);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = k.at(j) ? v[j] * a.d.scale : 0.f;
                }
                store8<T, VEC>(static_cast<T *>(a.dx) + r * a.lddx, c0, lane, a.cols, pack8<T>(v));
            }
        }
        fetch(r + S * groups, slot);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    if (a.part) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = col_of<VEC>((n * WARPS + wr) * kSeg, lane, j);
                if (c < a.cols)
                    a.part[g * (int64_t)a.cols + c] = dw[n][j];
            }
    }
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

template <typename T, bool VEC, int W, int N>
sg_status run_fwd(const NormFwd &a, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    constexpr int S = VEC ? ring_rows<T, 2, W, N>(fwd_ctas(W, N, sizeof(T))) : 1;
    constexpr int smem = VEC ? Ring8<T, 2, N, S, norm_threads(W)>::kBytes : 0;
    if constexpr (smem > 226 << 10) {  // fp32 rows above 16384 columns: not one is held
        return run_fwd<T, false, W, N>(a, st);
    } else {
        // Half the CTAs where only 16-bit rows are written and none of dropout's
        // work waits to be hidden: memory takes the rows faster the fewer are
        // read and written at a time, while two segments to a thread are enough
        // under way (16384 x 4096 bf16: 81 us, 97 with all; with dropout 104, 96;
        // to 8 bits 82, 75; 32768 x 1024, one segment: 55, 49).  Rows that fit
        // the L2 cache take all (1024 x 4096: 7.9 us, 8.5 with half).
        constexpr int kCtas = fwd_ctas(W, N, sizeof(T));
        const bool half = VEC && sizeof(T) == 2 && N > 1 && kCtas > 1 && !a.y8 && !a.d.drop &&
                          a.nrows * a.cols >= 8 << 20;  // 64 MB in and out
        const int64_t need = W == 1 ? ceil_div(a.nrows, 8) : a.nrows, most = kSMs * (half ? kCtas / 2 : kCtas);
        NORM_TRY(allow_smem(k_norm_fwd<T, VEC, W, N, S>, smem, done));
        k_norm_fwd<T, VEC, W, N, S><<<(unsigned)(need < most ? need : most), norm_threads(W), smem, st>>>(a);
        return SG_OK;
    }
}

template <typename T, bool VEC, int W, int N>
sg_status run_bwd(const NormBwd &a, int64_t grid, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    constexpr int S = VEC ? ring_rows<T, 3, W, N>(bwd_ctas(true, W, sizeof(T))) : 1;
    constexpr int smem = VEC ? Ring8<T, 3, N, S, norm_threads(W)>::kBytes : 0;
    if constexpr (smem > 226 << 10) {  // fp32 rows above 16384 columns: not one is held
        return run_bwd<T, false, W, N>(a, grid, st);
    } else {
        NORM_TRY(allow_smem(k_norm_bwd<T, VEC, W, N, S>, smem, done));
        k_norm_bwd<T, VEC, W, N, S><<<(unsigned)grid, norm_threads(W), smem, st>>>(a);
        return SG_OK;
    }
}

template <typename T, bool VEC>
sg_status launch_fwd(const NormFwd &a, cudaStream_t st)
{
    // 513 to 768 columns: one warp to a row leaves none of its lanes without
    // work and needs no barrier, but takes twice as long for one row.  65536 x
    // 768 bf16 to 8 bits with dropout: 68 us, 101 by four warps; 128 rows: 4.7
    // and 2.4 us.  So it is taken when there are rows for all warps.
    if (VEC && a.cols > 2 * kSeg && a.cols <= 3 * kSeg && a.nrows >= (int64_t)kSMs * fwd_ctas(1, 3, sizeof(T)) * 8)
        return run_fwd<T, VEC, 1, 3>(a, st);
#define X(W, N)                             \
    if (a.cols <= (int64_t)(W) * (N) * kSeg) \
        return run_fwd<T, VEC, W, N>(a, st);
    NORM_SHAPES(X)
#undef X
    return SG_ERR_UNSUPPORTED;  // not reached: cols <= kMaxCols
}

template <typename T, bool VEC>
sg_status launch_bwd(const NormBwd &a, int64_t grid, cudaStream_t st)
{
#define X(W, N)                             \
    if (a.cols <= (int64_t)(W) * (N) * kSeg) \
        return run_bwd<T, VEC, W, N>(a, grid, st);
    if constexpr (VEC) {
        NORM_SHAPES_BWD8(X)
    } else {
        NORM_SHAPES(X)
    }
#undef X
    return SG_ERR_UNSUPPORTED;  // not reached: cols <= kMaxCols
}

// CTAs of the backward kernel, and the row groups they make
int64_t bwd_groups(bool vec, int64_t nrows, int64_t cols, int size, int64_t *grid)
{
    int warps = 32;
#define X(W, N)                                           \
    if (warps == 32 && cols <= (int64_t)(W) * (N) * kSeg) \
        warps = (W);
    if (vec) {
        NORM_SHAPES_BWD8(X)
    } else {
        NORM_SHAPES(X)
    }
#undef X
    const int64_t need = warps == 1 ? ceil_div(nrows, 8) : nrows, most = kSMs * bwd_ctas(vec, warps, size);
    *grid = need < most ? need : most;
    return warps == 1 ? *grid * 8 : *grid;
}

template <typename T>
void launch_dropout(bool vec, const void *x, int64_t ldx, int64_t nrows, int64_t cols, const Drop &d, void *y,
                    int64_t ldy, cudaStream_t st)
{
    const T *xs = static_cast<const T *>(x);
    T *ys = static_cast<T *>(y);
    if (!vec) {
        const int64_t segs = ceil_div(cols, kSeg), slab = ((1ll << 31) - 1) / segs;  // rows of a launch
        for (int64_t r0 = 0; r0 < nrows; r0 += slab) {
            const int64_t n = (nrows - r0 < slab ? nrows - r0 : slab) * segs;
            k_dropout_any<T><<<(unsigned)ceil_div(n, kDropThreads / 32), kDropThreads, 0, st>>>(
                xs + r0 * ldx, ldx, (uint32_t)n, (uint32_t)segs, (int)cols, (uint32_t)r0, d, ys + r0 * ldy, ldy);
        }
        return;
    }
    // i / blks = (i magic) >> (32 + shift) for i < 2^31, with magic =
    // ceil(2^(32 + shift) / blks) and 2^shift < blks <= 2^(shift + 1): the
    // excess of magic, below blks / 2^(32 + shift) of 1 / blks, times i stays
    // below 1 / blks
    const uint32_t blks = (uint32_t)(cols / 8);
    uint32_t shift = 0;
    while ((2ull << shift) < blks)
        ++shift;
    const uint32_t magic = blks == 1 ? 0 : (uint32_t)(((1ull << (32 + shift)) + blks - 1) / blks);
    constexpr int U = drop_u(sizeof(T));
    const int64_t slab = ((1ll << 31) - 1 - kDropThreads * U) / blks;  // rows of a launch
    for (int64_t r0 = 0; r0 < nrows; r0 += slab) {
        const int64_t n = (nrows - r0 < slab ? nrows - r0 : slab) * blks;
        const unsigned grid = (unsigned)ceil_div(n, kDropThreads * U);
        if (ldx == cols && ldy == cols)
            k_dropout<T, true><<<grid, kDropThreads, 0, st>>>(xs + r0 * ldx, ldx, (uint32_t)n, blks, magic, shift,
                                                              (uint32_t)r0, d, ys + r0 * ldy, ldy);
        else
            k_dropout<T, false><<<grid, kDropThreads, 0, st>>>(xs + r0 * ldx, ldx, (uint32_t)n, blks, magic, shift,
                                                               (uint32_t)r0, d, ys + r0 * ldy, ldy);
    }
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
    NORM_TRY(check_vec(fn, "rstd", rstd));
    NORM_TRY(check_vec(fn, "y8_scale", y8_scale));
    NormFwd a;
    if (!make_drop(drop_p, seed, offset, &a.d))
        NORM_FAIL(SG_ERR_INVALID, "%s: drop_p=%g is not a probability", fn, drop_p);
    if (rows == 0)
        return SG_OK;
    a.x = x, a.res = residual, a.w = weight, a.u = u, a.y = y, a.y8 = y8, a.rstd = rstd, a.scale8 = y8_scale;
    a.ldx = ldx, a.ldr = ldr, a.ldu = ldu, a.ldy = ldy, a.ld8 = ldy8, a.nrows = rows, a.cols = (int)cols;
    a.eps = (float)eps;
    cudaStream_t st = (cudaStream_t)stream;
    // 8-bit rows are written in pieces of 8 bytes
    const bool vec = cols % 8 == 0 && vec_ok(x, ldx, es) && vec_ok(residual, ldr, es) && vec_ok(weight, cols, es) &&
                     vec_ok(u, ldu, es) && vec_ok(y, ldy, es) && (!y8 || (((uintptr_t)y8) % 8 == 0 && ldy8 % 8 == 0));
    if (dtype == SG_BF16)
        NORM_TRY((vec ? launch_fwd<__nv_bfloat16, true>(a, st) : launch_fwd<__nv_bfloat16, false>(a, st)));
    else if (dtype == SG_F16)
        NORM_TRY((vec ? launch_fwd<__half, true>(a, st) : launch_fwd<__half, false>(a, st)));
    else
        NORM_TRY((vec ? launch_fwd<float, true>(a, st) : launch_fwd<float, false>(a, st)));
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
    int64_t most = 0;  // groups of any type and mapping
    for (int i = 0; i < 4; ++i) {
        const int64_t n = bwd_groups(i & 1, rows, cols, i & 2 ? 2 : 4, &grid);
        most = n > most ? n : most;
    }
    *bytes = most * cols * 4;
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
    NORM_TRY(check_vec(fn, "rstd", rstd));
    NORM_TRY(check_vec(fn, "dweight", dweight));
    NormBwd a;
    if (!make_drop(drop_p, seed, offset, &a.d))
        NORM_FAIL(SG_ERR_INVALID, "%s: drop_p=%g is not a probability", fn, drop_p);
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        if (dweight)
            SG_TRY_CUDA(cudaMemsetAsync(dweight, 0, (size_t)cols * 4, st));
        return SG_OK;
    }
    const bool vec = cols % 8 == 0 && vec_ok(dy, lddy, es) && vec_ok(u, ldu, es) && vec_ok(du_in, lddu_in, es) &&
                     vec_ok(weight, cols, es) && vec_ok(du, lddu, es) && vec_ok(dx, lddx, es);
    int64_t grid;
    const int64_t groups = bwd_groups(vec, rows, cols, (int)es, &grid);
    if (dweight && (!work || work_bytes < groups * cols * 4 || ((uintptr_t)work) % 4 != 0))
        NORM_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_add_rmsnorm_bwd_work), aligned to 4", fn,
                  (long long)(groups * cols * 4));
    a.dy = dy, a.u = u, a.w = weight, a.du_in = du_in, a.rstd = rstd, a.du = du, a.dx = dx;
    a.part = dweight ? static_cast<float *>(work) : nullptr;
    a.lddy = lddy, a.ldu = ldu, a.ldi = lddu_in, a.ldo = lddu, a.lddx = lddx, a.nrows = rows, a.cols = (int)cols;
    if (dtype == SG_BF16)
        NORM_TRY((vec ? launch_bwd<__nv_bfloat16, true>(a, grid, st) : launch_bwd<__nv_bfloat16, false>(a, grid, st)));
    else if (dtype == SG_F16)
        NORM_TRY((vec ? launch_bwd<__half, true>(a, grid, st) : launch_bwd<__half, false>(a, grid, st)));
    else
        NORM_TRY((vec ? launch_bwd<float, true>(a, grid, st) : launch_bwd<float, false>(a, grid, st)));
    SG_TRY_CUDA(cudaGetLastError());
    if (dweight)
        return launch(cols < 2048 ? k_norm_dw<8> : k_norm_dw<32>,
                      dim3((unsigned)ceil_div(cols, cols < 2048 ? 8 : 32)), 1024, 0, 1, true, st,
                      (const float *)a.part, (int)groups, cols, dweight);
    return SG_OK;
}

}  // extern "C"
