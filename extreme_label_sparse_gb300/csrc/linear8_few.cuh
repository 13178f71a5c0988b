// The 8-bit linear layer's forward pass for at most 512 tokens: bound by reading
// W8, so its bytes are read once and brought to fp16 on the chip.
//
// Channels are the rows of the product: a tile has 128 of them, and out^T = W x^T
// has the tokens as columns, 128 of them to a tile.  TMA streams blocks of 128 x 128
// bytes of W8, and the tokens' bytes of the same K, through a ring of stages.  Teams
// of four warps take the blocks in turn: a thread has a channel, turns its 128 bytes
// into fp16 (a byte permutation and a subtraction for two) and stores them in tensor
// memory, from where the MMA reads its A operand; the tokens' bytes become fp16 rows
// in shared memory (128-byte swizzle), its B operand.  One thread issues the MMAs
// into one of two accumulators, epilogue warps add up the other one, of 1024 terms,
// in fp32 registers.
//
// The blocks of all tiles are cut into equal ranges for the SMs, so that all of
// them read to the end.  Tiles that a cut falls into are written as fp32 parts and
// joined in a fixed order by a small kernel; where whole tiles leave less idle
// time than that takes, the cuts go between tiles.
//
// Measured at 2048 x 128000 (262 MB): 16 tokens 49 us (5.3 TB/s; a block takes 750
// cycles, its bytes 700 at the copy rate), 48 tokens 53 us, 128 tokens 65 us (970
// cycles: the MMAs take 630 to issue).  4096 x 4096: 16 tokens 10.5 us, 128 tokens
// 17.8 us, of which the launches, the first loads and the join are the larger part.
#pragma once

#include "linear8_widen.cuh"

namespace {

constexpr int kBlockK = 128;   // bytes of K in a block
constexpr int kChunk = 8;      // blocks that are summed in tensor memory: 1024 terms
constexpr uint32_t kWTile = 128 * kBlockK;
constexpr int kMaxFew = 512;   // tokens that this way takes: their scales are in shared memory

// for up to TMAX tokens: stages, operand buffers, teams, epilogue warps
template <int TMAX>
struct Few {
    // The tokens are brought to fp16 by a launch before, and copied as they are:
    // with more than 64 of them turning their bytes into fp16 for each tile takes
    // longer than the tile's own (128 x 2048 x 128000: 101 us).
    static constexpr bool kWide = TMAX > 64;
    static constexpr int NS = TMAX <= 16 ? 10 : 6;
    static constexpr int NX = 3;  // stages of the wide tokens, which wait for their MMAs: apart from W's
    static constexpr int NB = 4;
    static constexpr int TEAMS = TMAX <= 64 ? 4 : 2;
    static constexpr int CW = 4 * TEAMS;  // warps that turn bytes into fp16
    static constexpr int EW = TMAX <= 16 ? 4 : 8;
    static constexpr int kCols = TMAX / (EW / 4);  // tokens of an epilogue thread
    static constexpr int kThreads = 32 * (CW + EW + 2 + kWide);
    static constexpr uint32_t kX = TMAX * kBlockK * 2;  // a buffer of the tokens in fp16
    static constexpr uint32_t kStage = kWTile + (kWide ? 0 : TMAX * kBlockK);
    static constexpr uint32_t kSmem = NS * kStage + (kWide ? NX : NB) * kX + 1024;
    static constexpr uint32_t kA = 2 * TMAX < 64 ? 64 : 2 * TMAX;  // first column of the A buffers, after D's
};

struct FewCtl {
    uint64_t full[10], empty[10], xfull[3], xempty[3], ready[4], freed[4], tfull[2], tempty[2];
    uint32_t tmem;
    int abort_flag;
    float xs[kMaxFew];
};

struct FewArgs {
    int32_t T, N, tn;     // tokens, channels, columns of the product (a multiple of 16)
    int32_t xb;           // rows of a box of the tokens
    int32_t tt;           // tiles of the tokens: above 128, of 128 each, and next to each other in the list
    int32_t kb, tiles;    // blocks of a tile, tiles
    int32_t whole;        // ranges are whole tiles
    int32_t cuts;         // or each tile is cut into this many, if not 0
    int32_t ctas, per, more;  // ranges of `per` blocks (whole: tiles), the first `more` of one more
    int32_t otype;
    const float *xs, *ws;
    void *out;
    int64_t ldo;
    float *part;          // [slot][tn][128]
    int32_t *status;
};

// first block of CTA c's range
__host__ __device__ __forceinline__ int64_t range_at(const FewArgs &a, int c)
{
    if (a.cuts)
        return (int64_t)(c / a.cuts) * a.kb + a.kb * (c % a.cuts) / a.cuts;
    return ((int64_t)a.per * c + (c < a.more ? c : a.more)) * (a.whole ? a.kb : 1);
}

// A CTA's range, tile by tile: segments of blocks [k, k + n) of a tile
struct Segment {
    int tile, k, n;
};

__device__ __forceinline__ bool segment_at(const FewArgs &a, int64_t &b, int64_t end, Segment &s)
{
    if (b >= end)
        return false;
    s.tile = (int)(b / a.kb);
    s.k = (int)(b - (int64_t)s.tile * a.kb);
    s.n = (int)(end - b < a.kb - s.k ? end - b : a.kb - s.k);
    b += s.n;
    return true;
}

__device__ __forceinline__ void put(float *p, float z) { *p = z; }
__device__ __forceinline__ void put(__half *p, float z) { *p = __float2half_rn(z); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float z) { *p = __float2bfloat16_rn(z); }

// f with a pointer of the output's type to element `at`
template <typename F>
__device__ __forceinline__ void with_out(const FewArgs &a, int64_t at, F f)
{
    if (a.otype == SG_F32)
        f(static_cast<float *>(a.out) + at);
    else if (a.otype == SG_F16)
        f(static_cast<__half *>(a.out) + at);
    else
        f(static_cast<__nv_bfloat16 *>(a.out) + at);
}

template <int TMAX>
__global__ void __launch_bounds__(Few<TMAX>::kThreads, 1)
    k_few(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mx,
          const __grid_constant__ FewArgs a)
{
    using F = Few<TMAX>;
    constexpr int NS = F::NS, NB = F::NB, EW = F::EW, CW = F::CW;
    __shared__ FewCtl c;
    extern __shared__ uint8_t dsm[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    if (threadIdx.x == 0) {
        c.abort_flag = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&c.full[s]), 1);
            mbar_init(smem_u32(&c.empty[s]), 4);
        }
        for (int s = 0; s < F::NX; ++s) {
            mbar_init(smem_u32(&c.xfull[s]), 1);
            mbar_init(smem_u32(&c.xempty[s]), 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(smem_u32(&c.ready[b]), 4);
            mbar_init(smem_u32(&c.freed[b]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&c.tfull[b]), 1);
            mbar_init(smem_u32(&c.tempty[b]), EW);
        }
        fence_mbar_init();
    }
    if (warp == CW + EW + 1) {
        tmem_alloc(smem_u32(&c.tmem), 512);
        tmem_relinquish();
    }
    grid_wait();
    grid_go();
    for (int i = threadIdx.x; i < a.T; i += F::kThreads)
        c.xs[i] = a.xs[i];
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = c.tmem;
    volatile int *abort_flag = &c.abort_flag;
    int32_t *status = lin_status(a.status);
    const int64_t first = range_at(a, (int)blockIdx.x), end = range_at(a, (int)blockIdx.x + 1);
    const int nblocks = (int)(end - first);

    if (warp < CW) {
        // ---------------------------------------------------------- bytes to fp16
        const int team = warp >> 2, q = warp & 3, row = q * 32 + lane, tid = threadIdx.x & 127;
        for (int i = team; i < nblocks; i += F::TEAMS) {
            const int s = i % NS, b = i % NB;
            const uint32_t st = base + (uint32_t)s * F::kStage, xf = base + NS * F::kStage + (uint32_t)b * F::kX;
            // The operand buffer first: it is free when the MMAs of block i - NB are
            // done, which are issued in order, so the bytes of block i - NS, that
            // the stage had before, have arrived.  A team that waited for its stage
            // first could come to it while those were still on their way, and take
            // the barrier's phase before them for its own.
            static_assert(NB <= NS, "a stage is taken again after its buffer");
            if (!__all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&c.freed[b]), ((uint32_t)(i / NB) & 1u) ^ 1u, abort_flag, status)) ||
                !__all_sync(0xffffffffu, mbar_wait(smem_u32(&c.full[s]), (uint32_t)(i / NS) & 1u, abort_flag, status)))
                break;
            tc_fence_after();
            const uint8_t *src = dsm + (st - smem_u32(dsm));
            const uint32_t ta = tbase + F::kA + (uint32_t)b * 64 + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(src + row * 128 + (((4 * h + u) ^ (row & 7)) << 4));
                    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        r[u * 8 + 2 * j] = bytes_f16(in[j] ^ 0x80808080u, 0);
                        r[u * 8 + 2 * j + 1] = bytes_f16(in[j] ^ 0x80808080u, 1);
                    }
                }
                tmem_st32(ta + h * 32, r);
            }
            if constexpr (!F::kWide) {
                // the tokens: 16 bytes to a thread at a time, eight threads to a row
                uint8_t *dst = dsm + (xf - smem_u32(dsm));
                for (int e = tid; e < a.tn * 8; e += 128) {
                    const int t = e >> 3, u = e & 7;
                    const uint4 w = *reinterpret_cast<const uint4 *>(src + kWTile + t * 128 + ((u ^ (t & 7)) << 4));
                    uint8_t *at = dst + (u >> 2) * (a.tn * 128) + t * 128;
                    const int v = (u & 3) * 2;
                    uint32_t p[8];
                    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[2 * j] = bytes_f16(in[j] ^ 0x80808080u, 0);
                        p[2 * j + 1] = bytes_f16(in[j] ^ 0x80808080u, 1);
                    }
                    // half of a row's threads begin with their second 16 bytes: the
                    // two halves' rows lie in the same banks
                    const bool odd = u >= 4;
                    const uint4 lo = make_uint4(p[0], p[1], p[2], p[3]), hi = make_uint4(p[4], p[5], p[6], p[7]);
                    *reinterpret_cast<uint4 *>(at + (((v + odd) ^ (t & 7)) << 4)) = odd ? hi : lo;
                    *reinterpret_cast<uint4 *>(at + (((v + !odd) ^ (t & 7)) << 4)) = odd ? lo : hi;
                }
            }
            tmem_st_wait();
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&c.empty[s]));
                mbar_arrive(smem_u32(&c.ready[b]));
            }
        }
    } else if (warp < CW + EW) {
        // ---------------------------------------------------------- epilogue
        // a thread has a channel and up to kCols tokens
        const int q = warp & 3, t0 = (warp - CW) / 4 * F::kCols;
        const int cols = min(F::kCols, a.tn - t0);  // a multiple of 16, or nothing to do
        int64_t b = first;
        Segment s;
        int it = 0;
        bool ok = true;
        while (ok && segment_at(a, b, end, s)) {
            const int n = s.tile / a.tt * 128 + q * 32 + lane, t1 = s.tile % a.tt * 128 + t0;  // the thread's first token
            const float ws = n < a.N ? a.ws[n] : 0.f;
            float v[F::kCols / 16][16] = {};
            for (int k = 0; k < s.n; k += kChunk, ++it) {
                const int buf = it & 1;
                ok = __all_sync(0xffffffffu,
                                mbar_wait(smem_u32(&c.tfull[buf]), (uint32_t)(it >> 1) & 1u, abort_flag, status));
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t tm = tbase + (uint32_t)(buf * TMAX + t0) + ((uint32_t)(q * 32) << 16);
#pragma unroll
                for (int cc = 0; cc < F::kCols / 16; ++cc) {
                    if (cc * 16 < cols) {
                        float w[16];
                        tmem_ld_chunk<16>(tm + cc * 16, w);
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            v[cc][x] += w[x];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&c.tempty[buf]));
            }
            if (!ok)
                break;
            if (s.n < a.kb) {
                // a part: the range's first if it does not begin its tile
                float *p = a.part + ((int64_t)(2 * blockIdx.x + (s.k == 0 ? 1 : 0)) * a.tn + t0) * 128 + q * 32 + lane;
#pragma unroll
                for (int cc = 0; cc < F::kCols / 16; ++cc)
                    if (cc * 16 < cols) {
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            p[(cc * 16 + x) * 128] = v[cc][x];
                    }
            } else if (n < a.N) {
                with_out(a, t1 * a.ldo + n, [&](auto *p) {
#pragma unroll
                    for (int cc = 0; cc < F::kCols / 16; ++cc) {
#pragma unroll
                        for (int x = 0; x < 16; ++x, p += a.ldo)
                            if (t1 + cc * 16 + x < a.T)
                                put(p, v[cc][x] * c.xs[t1 + cc * 16 + x] * ws);
                        asm volatile("" ::: "memory");  // or the scales of all tokens are loaded first, and spilled
                    }
                });
            }
        }
    } else if (warp == CW + EW || warp == CW + EW + 2) {
        // ---------------------------------------------------------- producers
        // of W and the tokens' bytes, or (the second) of the wide tokens
        const bool xs = warp != CW + EW;
        const int ns = xs ? F::NX : NS;
        int64_t b = first;
        Segment s;
        Ring r;
        bool ok = true;
        const uint32_t bytes = xs ? (uint32_t)a.xb * kBlockK * 2 : kWTile + (F::kWide ? 0 : (uint32_t)a.xb * kBlockK);
        while (ok && segment_at(a, b, end, s))
            for (int k = s.k; k < s.k + s.n; ++k, r.next(ns)) {
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(xs ? &c.xempty[r.i] : &c.empty[r.i]), r.ph ^ 1u,
                                                       abort_flag, status));
                if (!ok)
                    break;
                if (elect_one()) {
                    const uint32_t bar = smem_u32(xs ? &c.xfull[r.i] : &c.full[r.i]);
                    mbar_arrive_expect_tx(bar, bytes);
                    if (xs) {
                        const uint32_t st = base + NS * F::kStage + (uint32_t)r.i * F::kX;
                        const int t1 = s.tile % a.tt * 128;
                        tma_load_2d(st, &mx, k * kBlockK, t1, bar);
                        tma_load_2d(st + TMAX * 128, &mx, k * kBlockK + 64, t1, bar);
                    } else {
                        const uint32_t st = base + (uint32_t)r.i * F::kStage;
                        tma_load_2d(st, &mW, k * kBlockK, s.tile / a.tt * 128, bar);
                        if constexpr (!F::kWide)
                            tma_load_2d(st + kWTile, &mx, k * kBlockK, 0, bar);
                    }
                }
                __syncwarp();
            }
        if (!ok && lane == 0) {
            // gave up: copies on their way land long before this
            const uint64_t t0 = global_ns();
            while (global_ns() - t0 < 1000000u) {
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- MMA
        const uint32_t idesc = idesc_f16(128, a.tn, 0, 0);
        int64_t b = first;
        Segment s;
        Ring r, rs;  // of the operand buffers, and of the wide tokens' stages
        int it = 0;
        bool ok = true;
        while (ok && segment_at(a, b, end, s)) {
            for (int k = 0; ok && k < s.n; ++it) {
                const int buf = it & 1, stop = min(s.n, k + kChunk);
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c.tempty[buf]), ((uint32_t)(it >> 1) & 1u) ^ 1u,
                                                       abort_flag, status));
                if (!ok)
                    break;
                tc_fence_after();
                for (int k0 = k; k < stop; ++k) {
                    ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c.ready[r.i]), r.ph, abort_flag, status));
                    if (!ok)
                        break;
                    tc_fence_after();
                    if constexpr (F::kWide) {
                        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c.xfull[rs.i]), rs.ph, abort_flag, status));
                        if (!ok)
                            break;
                    }
                    if (elect_one()) {
                        const uint32_t xf = base + NS * F::kStage + (uint32_t)(F::kWide ? rs.i : r.i) * F::kX;
                        const uint32_t atom = F::kWide ? TMAX * 128 : a.tn * 128;  // 64 of K
                        const OpDesc dx(xf, false);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts(tbase + buf * TMAX, tbase + F::kA + (uint32_t)r.i * 64 + ks * 8,
                                   dx.at((uint32_t)(ks >> 2) * (atom / 16), ks & 3), idesc,
                                   (k > k0 || ks > 0) ? 1u : 0u);
                        mma_commit(smem_u32(&c.freed[r.i]));
                        if constexpr (F::kWide)
                            mma_commit(smem_u32(&c.xempty[rs.i]));
                    }
                    __syncwarp();
                    r.next(NB);
                    rs.next(F::NX);
                }
                if (ok && elect_one())
                    mma_commit(smem_u32(&c.tfull[buf]));
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == CW + EW + 1) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// The parts of the tile that the cut before CTA `blockIdx.x + 1` falls into,
// where it is the tile's first cut: added in the order of K.  A thread has a
// channel and every 2 gridDim.y-th token; the loads of its parts are under way
// together.  The places are worked out once for a CTA (by every thread, the join
// of 48 x 2048 x 128000 took 10 us).
__global__ void __launch_bounds__(256) k_few_join(const __grid_constant__ FewArgs a)
{
    __shared__ int sm[2];
    const int c0 = (int)blockIdx.x;  // has the tile's first blocks
    if (threadIdx.x == 0) {
        const int64_t cut = range_at(a, c0 + 1), tile = cut / a.kb, stop = (tile + 1) * a.kb;
        int parts = 1;  // after the first
        while (c0 + 1 + parts < a.ctas && range_at(a, c0 + 1 + parts) < stop)
            ++parts;
        sm[0] = (int)tile;
        sm[1] = cut == tile * a.kb || range_at(a, c0) > tile * a.kb ? 0 : parts;
    }
    __syncthreads();
    grid_wait();
    const int lane = threadIdx.x & 127, n = sm[0] / a.tt * 128 + lane, t1 = sm[0] % a.tt * 128, parts = sm[1];
    if (parts == 0 || n >= a.N)
        return;
    const int step = 2 * a.tn * 128;
    const float ws = a.ws[n], *head = a.part + (int64_t)(2 * c0 + 1) * a.tn * 128 + lane;
    const float *rest = head + a.tn * 128;
#pragma unroll 2
    for (int t = (int)blockIdx.y * 2 + threadIdx.x / 128; t < min(a.tn, a.T - t1); t += 2 * gridDim.y) {
        float z = head[t * 128];
#pragma unroll 4
        for (int c = 0; c < parts; ++c)
            z += rest[(int64_t)c * step + t * 128];
        with_out(a, (t1 + t) * a.ldo + n, [&](auto *o) { put(o, z * a.xs[t1 + t] * ws); });
    }
}

FewArgs few_args(int64_t T, int64_t H, int64_t N)
{
    FewArgs a = {};
    a.T = (int32_t)T;
    a.N = (int32_t)N;
    a.tt = (int32_t)ceil_div(T, 128);
    a.tn = a.tt > 1 ? 128 : (int32_t)ceil_div(T, 16) * 16;
    a.xb = a.tt > 1 ? 128 : (int32_t)ceil_div(T, 8) * 8;
    a.kb = (int32_t)ceil_div(H, kBlockK);
    a.tiles = (int32_t)ceil_div(N, 128) * a.tt;
    // Whole tiles where they keep the last SM less than nine blocks (about 4 us)
    // longer than equal ranges would.  Whole / equal: 6 blocks longer (48 x 1024 x 65536)
    // 19.8 / 22.4 us, 8 (16 x 1024 x 60000) 16.7 / 17.5; the two meet above the limit
    // (10 blocks, 48 x 1280 x 40000: 18.1 / 19.1, 11, 16 x 2048 x 65536: 29.1 / 29.9).
    a.whole = ceil_div(a.tiles, kSMs) * a.kb - (int64_t)a.tiles * a.kb / kSMs < 9;
    // Few tiles of many tokens, whose parts are large: each tile cut into as many
    // ranges, where those are at most two blocks longer than equal ones, most of
    // which lie in two tiles and end in two parts (128 x 4096 x 4096: 17.6 us, 18.7
    // with equal ranges; 64 tokens 12.8 and 11.5).
    const int64_t cuts = kSMs / a.tiles < a.kb ? kSMs / a.tiles : a.kb;
    if (T > 64 && !a.whole && cuts >= 2 && ceil_div(a.kb, cuts) <= (int64_t)a.tiles * a.kb / kSMs + 2) {
        a.cuts = (int32_t)cuts;
        a.ctas = (int32_t)(a.tiles * cuts);
        return a;
    }
    // at least one tile, or two blocks, to a range
    const int64_t n = a.whole ? a.tiles : (int64_t)a.tiles * a.kb, most = a.whole ? n : ceil_div(n, 2);
    a.ctas = (int32_t)(most < kSMs ? most : kSMs);
    a.per = (int32_t)(n / a.ctas);
    a.more = (int32_t)(n % a.ctas);
    return a;
}

template <int TMAX>
sg_status launch_few(const CUtensorMap &mW, const CUtensorMap &mx, const FewArgs &a, bool after, cudaStream_t st)
{
    // once for each device (one bit of the mask)
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    SG_TRY_CUDA(cudaGetDevice(&dev));
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        SG_TRY_CUDA(cudaFuncSetAttribute(k_few<TMAX>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Few<TMAX>::kSmem));
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch(k_few<TMAX>, dim3((unsigned)a.ctas), Few<TMAX>::kThreads, (int)Few<TMAX>::kSmem, 1, after, st, mW, mx, a);
}

// ---------------------------------------------------------------- a few rows by integer dot products
// One to four tokens: a warp has two channels, a lane every 32nd 16 bytes of
// their rows, and sums of up to kMostDot products in 32-bit integers are exact.
// Bound by reading W8: 1 x 2048 x 128000 takes 40.6 us (6.5 TB/s), 4 tokens 50 us
// (the integer products), 1 x 4096 x 4096 3 us.
constexpr int kDotTokens = 4;
constexpr int64_t kMostDot = (1 << 17) - 1;
constexpr int kDotRows = 2, kDotThreads = 256;

__device__ __forceinline__ int dot16(uint4 a, uint4 b, int s)
{
    s = __dp4a((int)a.x, (int)b.x, s);
    s = __dp4a((int)a.y, (int)b.y, s);
    s = __dp4a((int)a.z, (int)b.z, s);
    return __dp4a((int)a.w, (int)b.w, s);
}

// 16 bytes at column c < H of a row that starts anywhere: from the two aligned 16
// that they lie in, of which each that is read has a byte of the row.  Bytes past the
// last column may be anything.
template <bool STREAM>
__device__ __forceinline__ uint4 any16(const int8_t *row, int c, int H)
{
    const int off = (int)((uintptr_t)row & 15);  // the same for the warp
    const uint4 *at = reinterpret_cast<const uint4 *>(row + c - off);
    if (off == 0)
        return STREAM ? __ldcs(at) : *at;
    const uint4 a = at[0], b = c + 16 - off < H ? at[1] : make_uint4(0, 0, 0, 0);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8) {
#pragma unroll
        for (int j = 0; j < 6; ++j)
            w[j] = w[j + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int j = 0; j < 5; ++j)
            w[j] = w[j + 1];
    }
    const int s = 8 * (off & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                      __funnelshift_r(w[3], w[4], s));
}

// the first n bytes of 16, and 0
__device__ __forceinline__ uint4 first_bytes(uint4 v, int n)
{
    auto keep = [&](uint32_t w, int j) { return n >= 4 * j + 4 ? w : n <= 4 * j ? 0u : w & ((1u << (8 * (n - 4 * j))) - 1u); };
    return make_uint4(keep(v.x, 0), keep(v.y, 1), keep(v.z, 2), keep(v.w, 3));
}

// ANY: rows start anywhere (1 x 1001 x 32000: 14 us, copied to aligned rows first 21;
// 1 x 1024 x 32000, aligned: 6).
template <int TT, bool ANY>
__global__ void __launch_bounds__(kDotThreads)
    k_dot(const int8_t *__restrict__ x8, int64_t ldx, const int8_t *__restrict__ W8, int64_t ldw, int H,
          const __grid_constant__ FewArgs a)
{
    constexpr int U = 4;  // 16 bytes of a row under way together
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * (kDotThreads / 32) + threadIdx.x / 32) * kDotRows;
    grid_wait();
    grid_go();
    if (n0 >= a.N)
        return;
    const int8_t *w[kDotRows];
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)
        w[r] = W8 + (int64_t)min(n0 + r, a.N - 1) * ldw;
    auto load_w = [&](int r, int c) {
        if constexpr (ANY)
            return any16<true>(w[r], c, H);
        else
            return __ldcs(reinterpret_cast<const uint4 *>(w[r] + c));
    };
    auto load_x = [&](int t, int c) {
        if constexpr (ANY)
            return any16<false>(x8 + t * ldx, c, H);
        else
            return *reinterpret_cast<const uint4 *>(x8 + t * ldx + c);
    };
    int sum[kDotRows][TT] = {};
    int c = lane * 16;
    for (; c + (U - 1) * 512 + 16 <= H; c += U * 512) {
        uint4 v[kDotRows][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < kDotRows; ++r)
                v[r][u] = load_w(r, c + u * 512);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const uint4 x = t < a.T ? load_x(t, c + u * 512) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < kDotRows; ++r)
                    sum[r][t] = dot16(v[r][u], x, sum[r][t]);
            }
    }
    // the rest, whose last 16 may go past the row's end (not past its stride's 16):
    // what W has there meets zeros
    if (c < H) {
        uint4 v[kDotRows][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < kDotRows; ++r)
                if (c + u * 512 < H)
                    v[r][u] = load_w(r, c + u * 512);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = c + u * 512;
            if (at < H) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    uint4 x = t < a.T ? load_x(t, at) : make_uint4(0, 0, 0, 0);
                    if (at + 16 > H)
                        x = first_bytes(x, H - at);
#pragma unroll
                    for (int r = 0; r < kDotRows; ++r)
                        sum[r][t] = dot16(v[r][u], x, sum[r][t]);
                }
            }
        }
    }
    __syncwarp();
    int mine = 0;  // lane r TT + t has token t of channel n0 + r
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int z = __reduce_add_sync(0xffffffffu, sum[r][t]);
            mine = lane == r * TT + t ? z : mine;
        }
    const int t = lane % TT, n = n0 + lane / TT;
    if (lane < kDotRows * TT && t < a.T && n < a.N)
        with_out(a, t * a.ldo + n, [&](auto *p) { put(p, (float)mine * a.xs[t] * a.ws[n]); });
}

template <int TT, bool ANY>
sg_status launch_dot(const int8_t *x8, int64_t ldx, const int8_t *W8, int64_t ldw, int64_t H, const FewArgs &a,
                     bool after, cudaStream_t st)
{
    const int rows = kDotThreads / 32 * kDotRows;
    return launch(k_dot<TT, ANY>, dim3((unsigned)ceil_div(a.N, rows)), kDotThreads, 0, 1, after, st, x8, ldx, W8, ldw, (int)H, a);
}

// With many tokens W8 is better brought to 16 bits once, for the 16-bit products at
// twice the rate of k_few, which turns it into fp16 for each 128 tokens.  At 4096 x
// 4096 the two meet at some 700 tokens (512: 22.5 us this way, 30 the other; 640: 33 and
// 34; 768: 37 and 35), at 2048 x 65536 at a thousand (640: 141 and 191; 896: 195 and
// 225; 1024: 220 and 216).  kMaxFew stands below both.
bool is_few(int64_t T) { return T <= kMaxFew; }

bool by_dot(int64_t T, int64_t H) { return T <= kDotTokens && H <= kMostDot; }

// A call's work memory: fp32 parts, tokens (above 64 in fp16; else copies of rows
// that do not start on 16 bytes), and W8's rows that do not, in pieces of channels
struct FewPlan {
    int64_t Nc;              // channels of a piece
    int64_t ld;              // row stride of copies
    bool copy_x, copy_W;
    int64_t o_x, o_W, bytes;
};

constexpr int64_t kPiece = 256ll << 20;  // bytes of W8 in the work memory

int64_t few_parts(int64_t T, int64_t H, int64_t N)
{
    if (by_dot(T, H))
        return 0;
    const FewArgs a = few_args(T, H, N);
    return a.whole ? 0 : (int64_t)2 * kSMs * a.tn * 128 * 4;
}

FewPlan few_plan(const int8_t *x8, int64_t ldx, int64_t T, int64_t H, const int8_t *W8, int64_t ldw, int64_t N)
{
    FewPlan p = {};
    p.ld = ceil_div(H, 16) * 16;
    const bool any = by_dot(T, H) && T <= 2;  // k_dot takes such rows itself
    p.copy_x = !any && T <= 64 && !tma_ok(x8, ldx, 1);
    p.copy_W = !any && !tma_ok(W8, ldw, 1);
    p.Nc = N;
    if (p.copy_W && N * p.ld > kPiece) {
        p.Nc = kPiece / p.ld / 128 * 128;
        p.Nc = p.Nc < 128 ? 128 : p.Nc;
        p.Nc = p.Nc < N ? p.Nc : N;
    }
    auto take = [&](int64_t n) {
        const int64_t at = p.bytes;
        p.bytes += ceil_div(n, 256) * 256;
        return at;
    };
    const int64_t one = few_parts(T, H, p.Nc), rest = N % p.Nc ? few_parts(T, H, N % p.Nc) : 0;
    take(one > rest ? one : rest);
    p.o_x = take(T > 64 ? T * p.ld * 2 : p.copy_x ? T * p.ld : 0);
    p.o_W = take(p.copy_W ? p.Nc * p.ld : 0);
    return p;
}

sg_status few_fwd(const int8_t *x8, int64_t ldx, const float *xs, int64_t T, int64_t H, const int8_t *W8, int64_t ldw,
                  const float *ws, int64_t N, void *out, int64_t ldo, int32_t dtype, const FewPlan &p, uint8_t *work,
                  int32_t *status, cudaStream_t st)
{
    bool after = false;  // this call's kernels have begun
    if (T > 64) {
        LIN_TRY(widen(widen_of(x8, ldx, T, H, nullptr, 0, nullptr, work + p.o_x, p.ld, true), Widen{}, after, st));
        after = true;
    } else if (p.copy_x) {
        LIN_TRY(realign(x8, ldx, T, H, work + p.o_x, p.ld, after, st));
        after = true;
        x8 = reinterpret_cast<const int8_t *>(work + p.o_x);
        ldx = p.ld;
    }
    for (int64_t n0 = 0; n0 < N; n0 += p.Nc) {
        const int64_t nc = N - n0 < p.Nc ? N - n0 : p.Nc;
        const int8_t *W = W8 + n0 * ldw;
        int64_t ld = ldw;
        if (p.copy_W) {
            LIN_TRY(realign(W, ldw, nc, H, work + p.o_W, p.ld, after, st));
            after = true;
            W = reinterpret_cast<const int8_t *>(work + p.o_W);
            ld = p.ld;
        }
        FewArgs a = few_args(T, H, nc);
        a.otype = dtype;
        a.xs = xs, a.ws = ws + n0, a.ldo = ldo;
        a.out = static_cast<uint8_t *>(out) + n0 * (dtype == SG_F32 ? 4 : 2);
        a.part = reinterpret_cast<float *>(work);
        a.status = status;
        if (by_dot(T, H)) {
            const bool any = !tma_ok(x8, ldx, 1) || !tma_ok(W, ld, 1);
            LIN_TRY((T > 2    ? launch_dot<4, false>(x8, ldx, W, ld, H, a, after, st)
                     : T == 2 ? (any ? launch_dot<2, true> : launch_dot<2, false>)(x8, ldx, W, ld, H, a, after, st)
                              : (any ? launch_dot<1, true> : launch_dot<1, false>)(x8, ldx, W, ld, H, a, after, st)));
            after = true;
            continue;
        }
        CUtensorMap mW, mx;
        LIN_TRY(map_of(&mW, W, H, nc, ld, 1, "W8", 128));
        if (T > 64) {
            LIN_TRY(map_of(&mx, work + p.o_x, H, T, p.ld, 2, "x", (uint32_t)a.xb));
            LIN_TRY(launch_few<128>(mW, mx, a, after, st));
        } else {
            LIN_TRY(map_of(&mx, x8, H, T, ldx, 1, "x8", (uint32_t)a.xb));
            LIN_TRY(T <= 16 ? launch_few<16>(mW, mx, a, after, st) : launch_few<64>(mW, mx, a, after, st));
        }
        after = true;
        if (!a.whole && a.ctas > 1)
            LIN_TRY(launch(k_few_join, dim3((unsigned)a.ctas - 1, (unsigned)ceil_div(T < 128 ? T : 128, 8)), 256, 0, 1,
                           true, st, a));
    }
    return SG_OK;
}

}  // namespace
