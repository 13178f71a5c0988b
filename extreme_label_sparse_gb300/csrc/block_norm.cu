// The norms before and after a block, fused with its gate and the residual's
// scale (definitions in include/sg.h):
//   v = x rx post,  u = alpha residual + gate v,  y = u ru pre
// and the gradient through both.  Bound by memory, and by instructions where rows
// are turned into 8 bits or back: a row lies in the registers of one CTA (forward)
// or in shared memory (backward) between its two sums and their uses, so each input
// is read once and each output written once.  16384 x 4096 bf16: forward 84 us (6.4
// TB/s), with x kept in 8 bits 109, with u in 16 bits and y, x and u in 8, as a
// training step keeps them, 150 (its bytes take 89); backward 126 us (6.4 TB/s), from
// 8 bits 132 (5.1 TB/s).
#include <cmath>

#include "norm.cuh"
#include "quant8.cuh"

namespace {

constexpr int64_t kMaxBlockCols = 16384;

struct BlockFwd {
    const void *x, *res, *post, *gate, *pre;
    void *u, *y;
    int8_t *y8, *x8, *u8;
    float *rx, *ru, *y8_scale, *x8_scale, *u8_scale;
    int64_t ldx, ldr, ldu, ldy, ldy8, ldx8, ldu8, nrows;
    int cols;
    float alpha, eps;
};

constexpr int block_ctas(int warps) { return norm_ctas(warps, true); }

// gate post_weight and pre_weight of a thread's columns (0 past the last)
template <typename T, bool VEC, int WARPS, int NV>
__device__ __forceinline__ void block_weights(const void *post, const void *gate, const void *pre, int wr, int lane,
                                              int cols, float2 (&gp)[NV][4], float2 (&pw)[NV][4])
{
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c0 = (n * WARPS + wr) * kSeg;
        unpack4(load8<T, VEC>(static_cast<const T *>(pre), c0, lane, cols), pw[n]);
        unpack4(load8<T, VEC>(static_cast<const T *>(post), c0, lane, cols), gp[n]);
        if (gate) {
            float2 g[4];
            unpack4(load8<T, VEC>(static_cast<const T *>(gate), c0, lane, cols), g);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                gp[n][i] = mul2(gp[n][i], g[i]);
        }
    }
}

// A row by WARPS warps (one warp: eight rows to a CTA), NV segments to a warp;
// row groups step over the rows, with the next S rows on their way to shared
// memory.  Two segments to a thread and a row at a time: batches of rows, as the
// backward kernel has them, took 142 us for 16384 x 4096 bf16 with x kept in 8 bits
// (now 109), and four warps to a row of up to 1024 columns 146 us for 65536 x 768
// (two: 99).
template <typename T, bool VEC, int WARPS, int NV, int S>
__global__ void __launch_bounds__(norm_threads(WARPS), block_ctas(WARPS)) k_block_fwd(const BlockFwd a)
{
    __shared__ RowSums sm;
    extern __shared__ uint4 dyn[];
    const Ring8<T, 2, NV, S, norm_threads(WARPS)> ring(dyn);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int wr = WARPS == 1 ? 0 : warp;
    const int64_t groups = WARPS == 1 ? (int64_t)gridDim.x * 8 : (int64_t)gridDim.x;
    const int64_t g = WARPS == 1 ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
    const T *ax = static_cast<const T *>(a.x), *ar = static_cast<const T *>(a.res);
    // 1024 threads lack the registers for both ways to max |y| (4096 x 16384 bf16 to
    // 16 bits: 105 us, 112 with both, 101 with the third reduction alone)
    constexpr bool kThird = WARPS == 32;
    const int ng = (a.cols + kGroup - 1) / kGroup;
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
    float2 gp[NV][4], pre[NV][4];  // gate post_weight, pre_weight
    block_weights<T, VEC, WARPS, NV>(a.post, a.gate, a.pre, wr, lane, a.cols, gp, pre);
    auto col0 = [&](int n) { return (n * WARPS + wr) * kSeg; };
    int turn = 0, slot = 0;
    for (int64_t r = g; r < a.nrows; r += groups, turn += 2) {
        Pack8<T> p[NV];  // x, then u
        float2 ss = make_float2(0.f, 0.f);
        float none = 0.f;
        if constexpr (VEC)
            copies_wait<S - 1>();
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c0 = col0(n);
            float2 v[4];
            if constexpr (VEC) {
                if (c0 + lane * 8 < a.cols)
                    p[n] = ring.get(slot, 0, n);
                else
                    p[n] = pack8<T>({});
            } else {
                p[n] = load8<T, VEC>(ax + r * a.ldx, c0, lane, a.cols);
            }
            unpack4(p[n], v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ss = fma2(v[i], v[i], ss);
        }
        float sum = ss.x + ss.y;
        row_reduce<WARPS, false>(sum, none, sm, turn);
        if (a.x8)
            store_groups<T, VEC, NV>(
                p, lane, a.cols, [&](int) { return a.x8 + r * a.ldx8; }, [&](int) { return a.x8_scale + r * ng; }, col0);
        const float rx = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
        ss = make_float2(0.f, 0.f);
        uint32_t most = 0;  // of |u pre|
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c0 = col0(n);
            float2 v[4], w[4];
            unpack4(p[n], v);
            if (ar) {
                Pack8<T> t;
                if constexpr (VEC) {
                    if (c0 + lane * 8 < a.cols)
                        t = ring.get(slot, 1, n);
                    else
                        t = pack8<T>({});
                } else {
                    t = load8<T, VEC>(ar + r * a.ldr, c0, lane, a.cols);
                }
                unpack4(t, w);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = mul2(w[i], both(a.alpha));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = fma2(mul2(v[i], both(rx)), gp[n][i], w[i]);
            // the second norm is taken of the sum as it is stored, so that the
            // backward pass sees the same row
            p[n] = pack4<T>(v);
            unpack4(p[n], v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ss = fma2(v[i], v[i], ss);
            if (!kThird && a.y8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 t = mul2(v[i], pre[n][i]);
                    most = max(most, max(mag(t.x), mag(t.y)));
                }
            }
            if (a.u)
                store8<T, VEC>(static_cast<T *>(a.u) + r * a.ldu, c0, lane, a.cols, p[n]);
        }
        fetch(r + S * groups, slot);
        slot = slot + 1 == S ? 0 : slot + 1;
        float top = __uint_as_float(min(most, 0x7f800000u));  // NaN as infinity, which stays the largest
        sum = ss.x + ss.y;
        row_reduce<WARPS, true>(sum, top, sm, turn + 1);
        if (a.u8)
            store_groups<T, VEC, NV>(
                p, lane, a.cols, [&](int) { return a.u8 + r * a.ldu8; }, [&](int) { return a.u8_scale + r * ng; }, col0);
        const float ru = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
        if (lane == 0 && wr == 0) {
            if (a.rx)
                a.rx[r] = rx;
            if (a.ru)
                a.ru[r] = ru;
        }
        Scale8 s8 = {};
        if (a.y8) {
            // max |y|: where that is possible without a third reduction, ru max |u pre|.
            // Products that fp32 holds in a few bits or as infinity say too little of
            // y.  Products of 0 are below 2^-150, which leaves integers of 0 with ru
            // up to 2^22 (a quarter of a step of 2^-126): rows of zeros among them.
            float last = top * ru;
            const bool known = mag(top) - 0x00800000u < 0x7f000000u;  // from 2^-126, and finite
            if (kThird || (!known && !(top == 0.f && ru < 0x1p22f))) {
                most = 0;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    float2 y[4];
                    unpack4(p[n], y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = mul2(mul2(y[i], both(ru)), pre[n][i]);
                        most = max(most, max(mag(t.x), mag(t.y)));
                    }
                }
                last = __uint_as_float(min(most, 0x7f800000u));
                row_reduce<WARPS, true>(none, last, sm, turn);
                if constexpr (WARPS > 1)
                    __syncthreads();  // the next row's first sums use the same buffer
            }
            // a row whose sum is not finite has neither scale nor values
            s8 = scale8_of(mag(sum < INFINITY ? last : NAN));
            if (lane == 0 && wr == 0)
                a.y8_scale[r] = s8.scale;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c0 = col0(n);
            float2 y[4];
            unpack4(p[n], y);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = mul2(mul2(y[i], both(ru)), pre[n][i]);
            if (a.y)
                store8<T, VEC>(static_cast<T *>(a.y) + r * a.ldy, c0, lane, a.cols, pack4<T>(y));
            if (a.y8)
                store8q<VEC>(a.y8 + r * a.ldy8, c0, lane, a.cols, quant8(y, s8.inv));
        }
    }
}

struct BlockBwd {
    const void *dy, *u, *x, *du_in, *post, *gate, *pre;
    const float *u_scale, *x_scale, *rx, *ru;
    void *dres, *dx;
    float *part;  // [row groups][2][cols]: sums of dy m and of du h; or NULL
    int64_t lddy, ldu, ldx, ldi, ldo, lddx, nrows;
    int cols;
    float alpha;
};

// A thread's pieces of the next rows on their way to shared memory, as Ring8:
// dy and du_in, and x and u, or (HELD) their eight bytes and the scale of its
// group, which the lanes of a warp copy for each other in pieces of 16 bytes: after
// the wait for the copies comes a __syncwarp.  (Copies of each lane's own 8 bytes
// and scale: 155 us for 16384 x 4096.)
template <typename T, bool HELD, int NV, int THREADS>
struct BackRows {
    static constexpr int P = sizeof(Pack8<T>) / 16;
    static constexpr int k16 = HELD ? 2 * P : 4 * P;  // pieces of 16 bytes
    static constexpr int kScales = THREADS / 16;
    static constexpr int kPart = k16 * THREADS * 16 + (HELD ? 2 * (THREADS * 8 + kScales * 4) : 0);  // a segment's
    static constexpr int kRow = NV * kPart;
    uint8_t *base;

    __device__ __forceinline__ explicit BackRows(void *smem) : base(static_cast<uint8_t *>(smem)) {}
    __device__ __forceinline__ uint8_t *part(int slot, int n) const { return base + (slot * NV + n) * kPart; }
    __device__ __forceinline__ uint4 *at(int slot, int n, int piece) const
    {
        return reinterpret_cast<uint4 *>(part(slot, n)) + piece * THREADS + threadIdx.x;
    }
    __device__ __forceinline__ uint2 *at8(int slot, int n, int m) const
    {
        return reinterpret_cast<uint2 *>(part(slot, n) + k16 * THREADS * 16) + m * THREADS + threadIdx.x;
    }
    __device__ __forceinline__ float *scale(int slot, int n, int m) const
    {
        return reinterpret_cast<float *>(part(slot, n) + (k16 * 16 + 16) * THREADS) + m * kScales + threadIdx.x / 16;
    }
    // m: 0 dy, 1 du_in, 2 x, 3 u
    __device__ __forceinline__ void copy(int slot, int n, int m, const T *src) const
    {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t dst = tc::smem_u32(at(slot, n, m * P + i));
            if constexpr (P == 2)
                tc::cp_async16_l1(dst, reinterpret_cast<const uint4 *>(src) + i);
            else
                tc::cp_async16(dst, reinterpret_cast<const uint4 *>(src) + i);
        }
    }
    // A warp's segment that starts at column c0 of the rows x and u, and their
    // scales: half the lanes copy 16 bytes of the one, half of the other.
    __device__ __forceinline__ void copy8(int slot, int n, const int8_t *x, const float *xs, const int8_t *u,
                                          const float *us, int c0, int cols) const
    {
        const int lane = threadIdx.x & 31, m = lane >> 4, c = c0 + (lane & 15) * 16;
        if (c < cols) {
            const uint32_t d = tc::smem_u32(part(slot, n) + (k16 * 16 + m * 8) * THREADS) +
                               (threadIdx.x & ~31u) * 8 + (lane & 15) * 16;
            const int bytes = min(16, cols - c);  // the rest of the 16 is set to 0
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"((m ? u : x) + c), "r"(bytes)
                         : "memory");
        }
        // lanes 0 and 1: x's two groups, 2 and 3: u's
        const int at = c0 / kGroup + (lane & 1);
        if (lane < 4 && at * kGroup < cols)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                             tc::smem_u32(part(slot, n) + (k16 * 16 + 16) * THREADS) +
                             ((lane >> 1) * kScales + threadIdx.x / 32 * 2 + (lane & 1)) * 4),
                         "l"((lane >> 1 ? us : xs) + at)
                         : "memory");
    }
    __device__ __forceinline__ void get(int slot, int n, int m, float2 (&v)[4]) const
    {
        Pack8<T> p;
#pragma unroll
        for (int i = 0; i < P; ++i)
            reinterpret_cast<uint4 *>(&p)[i] = *at(slot, n, m * P + i);
        unpack4(p, v);
    }
};

// Eight values v s, s common to elements 0 to 3 (s0) and 4 to 7 (s1).  Rows held
// in 8 bits have the integers in v: their scales go into factors of the row.
struct Held {
    float2 v[4];
    float s0, s1;

    __device__ __forceinline__ float s(int i) const { return i < 2 ? s0 : s1; }
    // the sum of a b's elements, each times its s; ONE: there is one s
    template <bool ONE>
    __device__ __forceinline__ float dot(const float2 (&a)[4], const float2 (&b)[4]) const
    {
        float2 p = mul2(a[0], b[0]), q = mul2(a[2], b[2]);
        p = fma2(a[1], b[1], p);
        q = fma2(a[3], b[3], q);
        if constexpr (ONE) {
            p = add2(p, q);
            return s0 * (p.x + p.y);
        } else {
            return s0 * (p.x + p.y) + s1 * (q.x + q.y);
        }
    }
};

// Sums of each of R rows over the WARPS warps of a row group, as row_reduce.
template <int R>
struct BatchSums {
    float v[2][R][32];
};

template <int WARPS, int R>
__device__ __forceinline__ void batch_reduce(float (&a)[R], BatchSums<R> &sm, int turn)
{
    const int lane = threadIdx.x & 31;
    if constexpr (R == 4) {
        // the lanes take turns: after two steps a lane has one row, lane / 8's
        const bool hi = lane & 16, odd = lane & 8;
        float x = hi ? a[2] : a[0], y = hi ? a[3] : a[1];
        x += __shfl_xor_sync(0xffffffffu, hi ? a[0] : a[2], 16);
        y += __shfl_xor_sync(0xffffffffu, hi ? a[1] : a[3], 16);
        float z = odd ? y : x;
        z += __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            z += __shfl_xor_sync(0xffffffffu, z, o);
        if constexpr (WARPS > 1) {
            if ((lane & 7) == 0)
                sm.v[turn & 1][lane / 8][threadIdx.x / 32] = z;
            __syncthreads();
            const float *row = sm.v[turn & 1][lane / 8];
            z = (lane & 7) < WARPS ? row[lane & 7] : 0.f;
            if constexpr (WARPS > 8) {
#pragma unroll
                for (int w = 8; w < WARPS; w += 8)
                    z += row[w + (lane & 7)];
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
                z += __shfl_xor_sync(0xffffffffu, z, o);
        }
#pragma unroll
        for (int k = 0; k < R; ++k)
            a[k] = __shfl_sync(0xffffffffu, z, 8 * k);
        return;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < R; ++k)
            a[k] += __shfl_xor_sync(0xffffffffu, a[k], o);
    if constexpr (WARPS > 1) {
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < R; ++k)
                sm.v[turn & 1][k][threadIdx.x / 32] = a[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < R; ++k)
            a[k] = sm.v[turn & 1][k][threadIdx.x % WARPS];
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < R; ++k)
                a[k] += __shfl_xor_sync(0xffffffffu, a[k], o);
    }
}

// Row groups of WARPS warps step over batches of R rows: a row is a chain of two
// sums and three uses of its values, and R of them side by side hide the waits of
// each other (16384 x 4096 bf16 from 8 bits, one row at a time: 161 us).  The next
// batch is on its way to shared memory meanwhile.  A thread keeps the two sums of
// its columns in registers until its last row, and the groups' sums are joined by
// k_block_dw.
template <typename T, bool VEC, bool HELD, int WARPS, int NV, int R>
__global__ void __launch_bounds__(norm_threads(WARPS), block_ctas(WARPS)) k_block_bwd(const BlockBwd a)
{
    __shared__ BatchSums<R> sm;
    extern __shared__ uint4 dyn[];
    const BackRows<T, HELD, NV, norm_threads(WARPS)> rows(dyn);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int wr = WARPS == 1 ? 0 : warp;
    const int64_t groups = WARPS == 1 ? (int64_t)gridDim.x * 8 : (int64_t)gridDim.x;
    const int64_t g = WARPS == 1 ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
    const int ng = (a.cols + kGroup - 1) / kGroup;
    tc::grid_go();
    const T *ady = static_cast<const T *>(a.dy), *ai = static_cast<const T *>(a.du_in);
    // the batch of rows r0, r0 + groups, ... into half `half`
    auto fetch = [&](int64_t r0, int half) {
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int64_t r = r0 + k * groups;
                if (r >= a.nrows)
                    break;
                const int slot = half * R + k;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int c = (n * WARPS + wr) * kSeg + lane * 8;
                    if (c < a.cols) {
                        rows.copy(slot, n, 0, ady + r * a.lddy + c);
                        if (ai)
                            rows.copy(slot, n, 1, ai + r * a.ldi + c);
                        if constexpr (!HELD) {
                            rows.copy(slot, n, 2, static_cast<const T *>(a.x) + r * a.ldx + c);
                            rows.copy(slot, n, 3, static_cast<const T *>(a.u) + r * a.ldu + c);
                        }
                    }
                    if constexpr (HELD)
                        rows.copy8(slot, n, static_cast<const int8_t *>(a.x) + r * a.ldx, a.x_scale + r * ng,
                                   static_cast<const int8_t *>(a.u) + r * a.ldu, a.u_scale + r * ng,
                                   (n * WARPS + wr) * kSeg, a.cols);
                }
            }
            copies_commit();
        }
    };
    // rstd of the batch that begins with r0, row k's by lane k
    auto rstd_of = [&](const float *rstd, int64_t r0) {
        const int64_t r = r0 + lane * groups;
        return lane < R && r < a.nrows ? rstd[r] : 0.f;
    };
    fetch(g, 0);
    fetch(g + R * groups, 1);
    // gate post_weight and pre_weight, where 1024 threads leave no registers for
    // them read again for each use (4096 x 16384 bf16: 328 us with them spilled)
    constexpr bool kKeep = WARPS * NV < 64;
    float2 gp[kKeep ? NV : 1][4], pre[kKeep ? NV : 1][4];
    if constexpr (kKeep)
        block_weights<T, VEC, WARPS, NV>(a.post, a.gate, a.pre, wr, lane, a.cols, gp, pre);
    auto weights = [&](int n) {
        if constexpr (!kKeep)
            block_weights<T, VEC, 1, 1>(a.post, a.gate, a.pre, n * WARPS + wr, lane, a.cols, gp, pre);
        return kKeep ? n : 0;
    };
    float2 dpre[NV][4] = {}, dh[NV][4] = {};
    int turn = 0, half = 0;
    float next_u = rstd_of(a.ru, g), next_x = rstd_of(a.rx, g);
    for (int64_t r0 = g; r0 < a.nrows; r0 += R * groups, turn += 2, half ^= 1) {
        const float rus = next_u, rxs = next_x;
        next_u = rstd_of(a.ru, r0 + R * groups);
        next_x = rstd_of(a.rx, r0 + R * groups);
        // a row's values of this lane, again for each use (from shared memory, or,
        // without VEC, from the caches); rows past the last have rstd = 0, and
        // are left out where something is read or written
        auto dy_of = [&](int k, int n, int c0, float2 (&v)[4]) {
            if constexpr (VEC)
                rows.get(half * R + k, n, 0, v);
            else
                unpack4(load8<T, VEC>(ady + (r0 + k * groups) * a.lddy, c0, lane, a.cols), v);
        };
        // m: 0 x, 1 u
        auto held_of = [&](int k, int n, int c0, int m, const void *mat, int64_t ld, const float *scale, Held &h) {
            const int64_t r = r0 + k * groups;
            h.s0 = h.s1 = 1.f;
            if constexpr (VEC && HELD) {
                unquant8(*rows.at8(half * R + k, n, m), h.v);
                h.s0 = h.s1 = *rows.scale(half * R + k, n, m);
            } else if constexpr (VEC) {
                rows.get(half * R + k, n, 2 + m, h.v);
            } else if constexpr (HELD) {
                unquant8(load8q<VEC>(static_cast<const int8_t *>(mat) + r * ld, c0, lane, a.cols), h.v);
                const float *s = scale + r * ng + c0 / kGroup;
                h.s0 = c0 < a.cols ? s[0] : 0.f;
                h.s1 = c0 + kGroup < a.cols ? s[1] : 0.f;
            } else {
                unpack4(load8<T, VEC>(static_cast<const T *>(mat) + r * ld, c0, lane, a.cols), h.v);
            }
        };
        auto x_of = [&](int k, int n, int c0, Held &h) { held_of(k, n, c0, 0, a.x, a.ldx, a.x_scale, h); };
        auto u_of = [&](int k, int n, int c0, Held &h) { held_of(k, n, c0, 1, a.u, a.ldu, a.u_scale, h); };
        auto there = [&](int k) { return k == 0 || r0 + k * groups < a.nrows; };
        float dot[R], ru[R], rx[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            dot[k] = 0.f;
            ru[k] = __shfl_sync(0xffffffffu, rus, k);
            rx[k] = __shfl_sync(0xffffffffu, rxs, k);
        }
        if constexpr (VEC)
            copies_wait<1>();
        if constexpr (VEC && HELD)
            __syncwarp();
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!there(k))
                break;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int c0 = (n * WARPS + wr) * kSeg;
                if (VEC && c0 + lane * 8 >= a.cols)
                    break;  // and neither has a later segment columns of this thread
                const int m = weights(n);
                float2 t[4];
                Held u;
                dy_of(k, n, c0, t);
                u_of(k, n, c0, u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    t[i] = mul2(t[i], u.v[i]);
                    dpre[n][i] = fma2(t[i], both(ru[k] * u.s(i)), dpre[n][i]);
                }
                dot[k] += u.template dot<VEC || !HELD>(t, pre[m]);
            }
        }
        batch_reduce<WARPS, R>(dot, sm, turn);
        float2 du[R][NV][4];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!there(k))
                break;
            // as in the norm's own gradient: neither a square of u nor one of its
            // factor without the other, so that rows of any scale stay in range
            const float back_u = dot[k] / (float)a.cols * ru[k] * ru[k];
            dot[k] = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int c0 = (n * WARPS + wr) * kSeg;
                if (VEC && c0 + lane * 8 >= a.cols)
                    break;
                const int m = weights(n);
                float2 t[4];
                Held h;
                if (ai) {
                    if constexpr (VEC)
                        rows.get(half * R + k, n, 1, du[k][n]);
                    else
                        unpack4(load8<T, VEC>(ai + (r0 + k * groups) * a.ldi, c0, lane, a.cols), du[k][n]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        du[k][n][i] = make_float2(0.f, 0.f);
                }
                u_of(k, n, c0, h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // integers times (rstd s), which is about 1, in one factor
                    if constexpr (HELD)
                        du[k][n][i] = fma2(h.v[i], both(-back_u * (ru[k] * h.s(i))), du[k][n][i]);
                    else
                        du[k][n][i] = fma2(both(-back_u), mul2(h.v[i], both(ru[k])), du[k][n][i]);
                }
                dy_of(k, n, c0, t);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    du[k][n][i] = fma2(mul2(pre[m][i], both(ru[k])), t[i], du[k][n][i]);
                x_of(k, n, c0, h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    t[i] = mul2(du[k][n][i], h.v[i]);
                    dh[n][i] = fma2(t[i], both(rx[k] * h.s(i)), dh[n][i]);
                }
                dot[k] += h.template dot<VEC || !HELD>(t, gp[m]);
                if (a.dres) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        t[i] = mul2(du[k][n][i], both(a.alpha));
                    store8<T, VEC>(static_cast<T *>(a.dres) + (r0 + k * groups) * a.ldo, c0, lane, a.cols, pack4<T>(t));
                }
            }
        }
        batch_reduce<WARPS, R>(dot, sm, turn + 1);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!there(k))
                break;
            const float back_x = dot[k] / (float)a.cols * rx[k] * rx[k];
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int c0 = (n * WARPS + wr) * kSeg;
                if (VEC && c0 + lane * 8 >= a.cols)
                    break;
                const int m = weights(n);
                Held h;
                x_of(k, n, c0, h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 w = mul2(gp[m][i], both(rx[k]));
                    if constexpr (HELD)
                        h.v[i] = fma2(w, du[k][n][i], mul2(h.v[i], both(-back_x * (rx[k] * h.s(i)))));
                    else
                        h.v[i] = fma2(w, du[k][n][i], mul2(both(-back_x), mul2(h.v[i], both(rx[k]))));
                }
                store8<T, VEC>(static_cast<T *>(a.dx) + (r0 + k * groups) * a.lddx, c0, lane, a.cols, pack4<T>(h.v));
            }
        }
        if constexpr (VEC && HELD)
            __syncwarp();  // the scales are read by other lanes than copy them
        fetch(r0 + 2 * R * groups, half);
    }
    if (a.part) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = col_of<VEC>((n * WARPS + wr) * kSeg, lane, j);
                if (c < a.cols) {
                    a.part[g * 2 * (int64_t)a.cols + c] = j & 1 ? dpre[n][j / 2].y : dpre[n][j / 2].x;
                    a.part[(g * 2 + 1) * (int64_t)a.cols + c] = j & 1 ? dh[n][j / 2].y : dh[n][j / 2].x;
                }
            }
    }
}

// The column sums joined in a fixed order, as k_norm_dw: blockIdx.y 0 for dpre, 1
// for S = sum of du h, of which dpost = gate S and dgate = post S.
template <typename T, int NC>
__global__ void __launch_bounds__(1024)
    k_block_dw(const float *__restrict__ part, int nparts, int64_t cols, const T *__restrict__ post,
               const T *__restrict__ gate, float *__restrict__ dpost, float *__restrict__ dgate,
               float *__restrict__ dpre)
{
    __shared__ float sm[32][NC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * NC + lane % NC;
    float s = 0.f;
    tc::grid_wait();
    if (c < cols) {
#pragma unroll 4
        for (int i = threadIdx.x / NC; i < nparts; i += 1024 / NC)
            s += part[(2 * i + blockIdx.y) * cols + c];
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
        if (blockIdx.y == 0) {
            if (dpre)
                dpre[c] = s;
        } else {
            if (dpost)
                dpost[c] = s * (gate ? to_f(gate[c]) : 1.f);
            if (dgate)
                dgate[c] = s * to_f(post[c]);
        }
    }
}

#define BLOCK_SHAPES(X) X(1, 1) X(1, 2) X(2, 2) X(4, 2) X(8, 2) X(16, 2) X(32, 2)
// of the backward kernel: one segment to a thread leaves registers for batches
#define BLOCK_SHAPES_BWD(X) X(1, 1) X(2, 1) X(4, 1) X(8, 1) X(16, 1) X(16, 2) X(32, 2)

template <typename T, bool VEC, int W, int N>
sg_status run_fwd(const BlockFwd &a, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    constexpr int S = VEC ? ring_rows<T, 2, W, N>(block_ctas(W)) : 1;
    constexpr int smem = VEC ? Ring8<T, 2, N, S, norm_threads(W)>::kBytes : 0;
    const int64_t need = W == 1 ? ceil_div(a.nrows, 8) : a.nrows, most = kSMs * block_ctas(W);
    NORM_TRY(allow_smem(k_block_fwd<T, VEC, W, N, S>, smem, done));
    k_block_fwd<T, VEC, W, N, S><<<(unsigned)(need < most ? need : most), norm_threads(W), smem, st>>>(a);
    return SG_OK;
}

// rows of a batch: two batches are in shared memory at a time
template <typename T, bool HELD, int W, int N>
constexpr int back_rows()
{
    const int s = (216 << 10) / block_ctas(W) / (2 * BackRows<T, HELD, N, norm_threads(W)>::kRow);
    const int most = W >= 32 ? 1 : N > 1 ? 2 : 4;
    return s > most ? most : s < 1 ? 1 : s;
}

template <typename T, bool VEC, bool HELD, int W, int N>
sg_status run_bwd(const BlockBwd &a, int64_t grid, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    constexpr int R = VEC ? back_rows<T, HELD, W, N>() : N > 1 || W > 16 ? 1 : 2;
    constexpr int smem = VEC ? 2 * R * BackRows<T, HELD, N, norm_threads(W)>::kRow : 0;
    if constexpr (smem > 224 << 10) {  // rows of which not two are held: fp32 above 4096 columns, 16 bits above 8192
        return run_bwd<T, false, HELD, W, N>(a, grid, st);
    } else {
        NORM_TRY(allow_smem(k_block_bwd<T, VEC, HELD, W, N, R>, smem, done));
        k_block_bwd<T, VEC, HELD, W, N, R><<<(unsigned)grid, norm_threads(W), smem, st>>>(a);
        return SG_OK;
    }
}

template <typename T, bool VEC>
sg_status launch_fwd(const BlockFwd &a, cudaStream_t st)
{
#define X(W, N)                             \
    if (a.cols <= (int64_t)(W) * (N) * kSeg) \
        return run_fwd<T, VEC, W, N>(a, st);
    BLOCK_SHAPES(X)
#undef X
    return SG_ERR_UNSUPPORTED;  // not reached: cols <= kMaxBlockCols
}

template <typename T, bool VEC, bool HELD>
sg_status launch_bwd(const BlockBwd &a, int64_t grid, cudaStream_t st)
{
#define X(W, N)                             \
    if (a.cols <= (int64_t)(W) * (N) * kSeg) \
        return run_bwd<T, VEC, HELD, W, N>(a, grid, st);
    BLOCK_SHAPES_BWD(X)
#undef X
    return SG_ERR_UNSUPPORTED;  // not reached: cols <= kMaxBlockCols
}

// CTAs of the backward kernel, and the row groups they make
int64_t bwd_groups(int64_t nrows, int64_t cols, int64_t *grid)
{
    int warps = 0;
#define X(W, N)                                          \
    if (warps == 0 && cols <= (int64_t)(W) * (N) * kSeg) \
        warps = (W);
    BLOCK_SHAPES_BWD(X)
#undef X
    const int64_t need = warps == 1 ? ceil_div(nrows, 8) : nrows, most = kSMs * block_ctas(warps);
    *grid = need < most ? need : most;
    return warps == 1 ? *grid * 8 : *grid;
}

template <typename T>
sg_status backward(const BlockBwd &a, bool vec, int64_t grid, int64_t groups, float *dpost, float *dgate, float *dpre,
                   cudaStream_t st)
{
    if (a.u_scale)
        NORM_TRY((vec ? launch_bwd<T, true, true>(a, grid, st) : launch_bwd<T, false, true>(a, grid, st)));
    else
        NORM_TRY((vec ? launch_bwd<T, true, false>(a, grid, st) : launch_bwd<T, false, false>(a, grid, st)));
    SG_TRY_CUDA(cudaGetLastError());
    if (!a.part)
        return SG_OK;
    const bool few = a.cols < 2048;
    return launch(few ? k_block_dw<T, 8> : k_block_dw<T, 32>, dim3((unsigned)ceil_div(a.cols, few ? 8 : 32), 2), 1024,
                  0, 1, true, st, (const float *)a.part, (int)groups, (int64_t)a.cols, static_cast<const T *>(a.post),
                  static_cast<const T *>(a.gate), dpost, dgate, dpre);
}

sg_status check_block(const char *fn, int64_t nrows, int64_t cols, int32_t dtype, const void *post, const void *gate,
                      const void *pre, double residual_scale)
{
    NORM_TRY(check_rows(fn, nrows, cols, dtype));
    if (cols > kMaxBlockCols)
        NORM_FAIL(SG_ERR_UNSUPPORTED, "%s: cols=%lld is above %lld", fn, (long long)cols, (long long)kMaxBlockCols);
    if (!post || !pre)
        NORM_FAIL(SG_ERR_INVALID, "%s: a weight is NULL (post_weight, pre_weight)", fn);
    if (!std::isfinite((float)residual_scale))
        NORM_FAIL(SG_ERR_INVALID, "%s: residual_scale=%g is not a finite fp32 number", fn, residual_scale);
    const int64_t es = elem_size(dtype);
    NORM_TRY(check_mat(fn, "post_weight", post, cols, cols, es));
    NORM_TRY(check_mat(fn, "gate", gate, cols, cols, es));
    return check_mat(fn, "pre_weight", pre, cols, cols, es);
}

}  // namespace

extern "C" {

sg_status sg_block_norm_fwd(const void *x, int64_t ldx, const void *residual, int64_t ldr, int64_t rows, int64_t cols,
                            int32_t dtype, const void *post_weight, const void *gate, const void *pre_weight,
                            double residual_scale, double eps, void *u, int64_t ldu, float *rstd_x, float *rstd_u,
                            void *y, int64_t ldy, int8_t *y8, int64_t ldy8, float *y8_scale, int8_t *x8, int64_t ldx8,
                            float *x8_scale, int8_t *u8, int64_t ldu8, float *u8_scale, void *stream)
{
    const char *fn = "sg_block_norm_fwd";
    NvtxRange nvtx_(fn);
    NORM_TRY(check_block(fn, rows, cols, dtype, post_weight, gate, pre_weight, residual_scale));
    if (rows && (!x || (!y && !y8)))
        NORM_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL (x, y or y8)", fn);
    if (rows && ((y8 && !y8_scale) || (x8 && !x8_scale) || (u8 && !u8_scale)))
        NORM_FAIL(SG_ERR_INVALID, "%s: 8-bit rows need their scales", fn);
    if (!(eps >= 0.0) || !std::isfinite(eps))
        NORM_FAIL(SG_ERR_INVALID, "%s: eps=%g is not a finite number >= 0", fn, eps);
    const int64_t es = elem_size(dtype);
    NORM_TRY(check_mat(fn, "x", x, ldx, cols, es));
    NORM_TRY(check_mat(fn, "residual", residual, ldr, cols, es));
    NORM_TRY(check_mat(fn, "u", u, ldu, cols, es));
    NORM_TRY(check_mat(fn, "y", y, ldy, cols, es));
    NORM_TRY(check_mat(fn, "y8", y8, ldy8, cols, 1));
    NORM_TRY(check_mat(fn, "x8", x8, ldx8, cols, 1));
    NORM_TRY(check_mat(fn, "u8", u8, ldu8, cols, 1));
    NORM_TRY(check_vec(fn, "rstd_x", rstd_x));
    NORM_TRY(check_vec(fn, "rstd_u", rstd_u));
    NORM_TRY(check_vec(fn, "y8_scale", y8_scale));
    NORM_TRY(check_vec(fn, "x8_scale", x8_scale));
    NORM_TRY(check_vec(fn, "u8_scale", u8_scale));
    if (rows == 0)
        return SG_OK;
    BlockFwd a;
    a.x = x, a.res = residual, a.post = post_weight, a.gate = gate, a.pre = pre_weight, a.u = u, a.y = y;
    a.y8 = y8, a.x8 = x8, a.u8 = u8, a.rx = rstd_x, a.ru = rstd_u;
    a.y8_scale = y8_scale, a.x8_scale = x8_scale, a.u8_scale = u8_scale;
    a.ldx = ldx, a.ldr = ldr, a.ldu = ldu, a.ldy = ldy, a.ldy8 = ldy8, a.ldx8 = ldx8, a.ldu8 = ldu8;
    a.nrows = rows, a.cols = (int)cols, a.alpha = (float)residual_scale, a.eps = (float)eps;
    cudaStream_t st = (cudaStream_t)stream;
    const bool vec = cols % 8 == 0 && vec_ok(x, ldx, es) && vec_ok(residual, ldr, es) && vec_ok(post_weight, cols, es) &&
                     vec_ok(gate, cols, es) && vec_ok(pre_weight, cols, es) && vec_ok(u, ldu, es) &&
                     vec_ok(y, ldy, es) && vec8_ok(y8, ldy8) && vec8_ok(x8, ldx8) && vec8_ok(u8, ldu8);
    if (dtype == SG_BF16)
        NORM_TRY((vec ? launch_fwd<__nv_bfloat16, true>(a, st) : launch_fwd<__nv_bfloat16, false>(a, st)));
    else if (dtype == SG_F16)
        NORM_TRY((vec ? launch_fwd<__half, true>(a, st) : launch_fwd<__half, false>(a, st)));
    else
        NORM_TRY((vec ? launch_fwd<float, true>(a, st) : launch_fwd<float, false>(a, st)));
    SG_TRY_CUDA(cudaGetLastError());
    return SG_OK;
}

sg_status sg_block_norm_bwd_work(int64_t rows, int64_t cols, int64_t *bytes)
{
    const char *fn = "sg_block_norm_bwd_work";
    if (!bytes)
        NORM_FAIL(SG_ERR_INVALID, "%s: bytes is NULL", fn);
    NORM_TRY(check_rows(fn, rows, cols, SG_F32));
    if (cols > kMaxBlockCols)
        NORM_FAIL(SG_ERR_UNSUPPORTED, "%s: cols=%lld is above %lld", fn, (long long)cols, (long long)kMaxBlockCols);
    int64_t grid;
    *bytes = bwd_groups(rows, cols, &grid) * 2 * cols * 4;
    return SG_OK;
}

sg_status sg_block_norm_bwd(const void *dy, int64_t lddy, const void *u, int64_t ldu, const float *u_scale,
                            const void *x, int64_t ldx, const float *x_scale, const void *du_in, int64_t lddu_in,
                            int64_t rows, int64_t cols, int32_t dtype, const void *post_weight, const void *gate,
                            const void *pre_weight, double residual_scale, const float *rstd_x, const float *rstd_u,
                            void *dresidual, int64_t lddr, void *dx, int64_t lddx, float *dpost, float *dgate,
                            float *dpre, void *work, int64_t work_bytes, void *stream)
{
    const char *fn = "sg_block_norm_bwd";
    NvtxRange nvtx_(fn);
    NORM_TRY(check_block(fn, rows, cols, dtype, post_weight, gate, pre_weight, residual_scale));
    if (rows && (!dy || !u || !x || !rstd_x || !rstd_u || !dx))
        NORM_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL (dy, u, x, rstd_x, rstd_u, dx)", fn);
    if (!u_scale != !x_scale)
        NORM_FAIL(SG_ERR_INVALID, "%s: x and u are both held in 8 bits, with their scales, or neither", fn);
    if (dgate && !gate)
        NORM_FAIL(SG_ERR_INVALID, "%s: dgate without a gate", fn);
    const int64_t es = elem_size(dtype), hs = u_scale ? 1 : es;
    NORM_TRY(check_mat(fn, "dy", dy, lddy, cols, es));
    NORM_TRY(check_mat(fn, "u", u, ldu, cols, hs));
    NORM_TRY(check_mat(fn, "x", x, ldx, cols, hs));
    NORM_TRY(check_mat(fn, "du_in", du_in, lddu_in, cols, es));
    NORM_TRY(check_mat(fn, "dresidual", dresidual, lddr, cols, es));
    NORM_TRY(check_mat(fn, "dx", dx, lddx, cols, es));
    NORM_TRY(check_vec(fn, "u_scale", u_scale));
    NORM_TRY(check_vec(fn, "x_scale", x_scale));
    NORM_TRY(check_vec(fn, "rstd_x", rstd_x));
    NORM_TRY(check_vec(fn, "rstd_u", rstd_u));
    NORM_TRY(check_vec(fn, "dpost", dpost));
    NORM_TRY(check_vec(fn, "dgate", dgate));
    NORM_TRY(check_vec(fn, "dpre", dpre));
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        for (float *d : {dpost, dgate, dpre})
            if (d)
                SG_TRY_CUDA(cudaMemsetAsync(d, 0, (size_t)cols * 4, st));
        return SG_OK;
    }
    const bool sums = dpost || dgate || dpre;
    auto vec16_ok = [](const void *m, int64_t ld) { return ((uintptr_t)m & 15) == 0 && ld % 16 == 0; };
    const bool held_ok = u_scale ? vec16_ok(u, ldu) && vec16_ok(x, ldx) : vec_ok(u, ldu, es) && vec_ok(x, ldx, es);
    const bool vec = cols % 8 == 0 && held_ok && vec_ok(dy, lddy, es) && vec_ok(du_in, lddu_in, es) &&
                     vec_ok(post_weight, cols, es) && vec_ok(gate, cols, es) && vec_ok(pre_weight, cols, es) &&
                     vec_ok(dresidual, lddr, es) && vec_ok(dx, lddx, es);
    int64_t grid;
    const int64_t groups = bwd_groups(rows, cols, &grid), need = groups * 2 * cols * 4;
    if (sums && (!work || work_bytes < need || ((uintptr_t)work) % 4 != 0))
        NORM_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_block_norm_bwd_work), aligned to 4", fn,
                  (long long)need);
    BlockBwd a;
    a.dy = dy, a.u = u, a.x = x, a.du_in = du_in, a.post = post_weight, a.gate = gate, a.pre = pre_weight;
    a.u_scale = u_scale, a.x_scale = x_scale, a.rx = rstd_x, a.ru = rstd_u, a.dres = dresidual, a.dx = dx;
    a.part = sums ? static_cast<float *>(work) : nullptr;
    a.lddy = lddy, a.ldu = ldu, a.ldx = ldx, a.ldi = lddu_in, a.ldo = lddr, a.lddx = lddx;
    a.nrows = rows, a.cols = (int)cols, a.alpha = (float)residual_scale;
    if (dtype == SG_BF16)
        return backward<__nv_bfloat16>(a, vec, grid, groups, dpost, dgate, dpre, st);
    if (dtype == SG_F16)
        return backward<__half>(a, vec, grid, groups, dpost, dgate, dpre, st);
    return backward<float>(a, vec, grid, groups, dpost, dgate, dpre, st);
}

}  // extern "C"
