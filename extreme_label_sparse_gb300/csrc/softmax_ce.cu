// Softmax cross entropy over a large label set (definitions in include/sg.h):
//   z = h W^T,  lse_t = log sum_v exp z_tv,
//   loss_t = lse_t - (1 - e) z_t,y - e mean_v z_t,
//   g_tv = dloss_t (exp(z_tv - lse_t) - (1 - e) [v = y_t] - e / V),
//   dh = g W,  dW = g^T h.
// The logits never reach memory.  Forward: one matrix product whose epilogue
// reduces each tile of logits to a running maximum and sum per row; a small
// kernel joins them.  Backward: the vocabulary goes by in pieces.  The product
// is taken again, its epilogue turning a piece's logits into g (16 bits, a few
// pieces of it held at a time), and the two gradient products follow a few
// pieces behind, so that they find the piece's W and g in the L2 cache: all in
// one launch, whose CTAs wait for one another's pieces by counters.
//
// All three products share one kernel: a persistent CTA, or a pair of CTAs on
// one 256 x 256 tile where there are more than 128 rows, walks a list of
// tiles.  A producer warp streams 128-byte wide K blocks of A and B through a
// ring of shared-memory stages (TMA, 128-byte swizzle), one thread issues
// tcgen05.mma into one of two TMEM accumulators, and eight warps work on the
// other one.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdlib>

#include "sg_internal.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

using namespace tc;

namespace {

#define CE_FAIL(code, ...)         \
    do {                           \
        sg_set_error(__VA_ARGS__); \
        return code;               \
    } while (0)
#define CE_TRY(expr)            \
    do {                        \
        sg_status rc_ = (expr); \
        if (rc_ != SG_OK)       \
            return rc_;         \
    } while (0)

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kSMs = 152;
constexpr int kEpiWarps = 8;
constexpr int kCeThreads = 32 * (kEpiWarps + 4);
constexpr int kBN = 256;                 // tile columns
constexpr uint32_t kBox = 8192;          // one TMA box: 64 rows of 128 bytes
constexpr uint32_t kStgWarp = 32 * 17 * 4;  // an epilogue warp's 32 x 32 outputs, rows 4 bytes apart
constexpr int kBand = 16;                // row tiles that walk the vocabulary together

template <int CG>
struct Cfg {
    static constexpr int BM = 128 * CG;            // tile rows
    static constexpr int BRows = kBN / CG;         // rows of B in one CTA
    static constexpr uint32_t kA = 2 * kBox;       // bytes of A's and B's part of a stage
    static constexpr uint32_t kB = (BRows / 64) * kBox;
    static constexpr uint32_t kStage = kA + kB;
    static constexpr int NS = CG == 2 ? 6 : 4;
    static constexpr uint32_t kSmem = NS * kStage + kEpiWarps * kStgWarp + 1024;
};

enum Mode { kLse = 0, kBwd = 1 };

struct CeArgs {
    int32_t T, V, H;      // rows, vocabulary, features
    int32_t C;            // clusters of the launch
    int32_t nm, nn, nk;   // tiles of the logits (rows, columns; of a piece in kBwd), K blocks
    int32_t f16;          // 16-bit operands are fp16, not bf16
    const int32_t *targets;
    int32_t ignore;
    int32_t *status;
    // kLse
    const float *h_scale, *W_scale;  // fp8: scale per row, or NULL
    float2 *part;         // running maximum (of z log2 e) and sum: [row][slot] for one row tile, else [slot][row]
    float *zsum;          // the same for the sum of z, or NULL
    float *ztgt;          // [T] the target's logit
    int32_t Tp;
    // kBwd
    const float *lse, *dloss;
    float *gscale;        // factor of g and its inverse, written by the first CTA
    float smooth, full;   // full: see g_scale
    int32_t pieces, Vc, lag, ring;  // of the vocabulary; the gradients follow `lag` behind, g is held `ring` deep
    int32_t nh;           // tiles along H
    int32_t dh_tiles, dh_split, dh_units;  // tiles, pieces of K, their product (0: no dh)
    int32_t dw, dw_nk;    // dW wanted; K blocks
    int32_t dw_more;      // dW tiles that a cluster with one dh unit less takes before the others share the rest
    float *acc;           // dh sums, [unit][CTA][column / 4][128 rows][4]
    uint16_t *g, *dW;
    int64_t ldg, lddW;
    int32_t dw_align;     // bytes that dW's rows start on: 32, 16 or 2 (any)
    uint32_t *g_done, *w_done;  // for each piece: CTAs that have stored a tile of g, gradient tiles that have read it
};

struct Tile {
    int kind;  // 0: logits, 1: dh, 2: dW
    int m0, n0, k0, nk, unit, piece;
};

// The tiles of cluster c, in the order in which each of its warps takes them.
// In kBwd phase p has the logits of piece p and then the gradients of piece p -
// lag.  A dh unit stays with one cluster through all pieces, which adds to its
// sums in order; the other tiles go round the clusters, each kind going on
// from one piece to the next where it stopped.
template <int CG, int MODE>
struct Walk {
    uint32_t c, j = 0;
    int phase = 0, stage = 0;

    __device__ __forceinline__ explicit Walk(int cluster) : c((uint32_t)cluster) {}

    // the j-th of this cluster's tiles in a round that starts at tile `from` of
    // the kind
    __device__ __forceinline__ uint32_t turn(const CeArgs &a, uint32_t from) const
    {
        const uint32_t C = a.C, at = from % C;
        return (c >= at ? c - at : c + C - at) + j * C;
    }

    __device__ __forceinline__ bool next(const CeArgs &a, Tile &t)
    {
        constexpr int BM = Cfg<CG>::BM;
        if constexpr (MODE == kLse) {
            // bands of kBand row tiles; inside a band the row tile runs
            // fastest, so W is read from memory once for a band
            const uint32_t l = j++ * a.C + c;
            if (l >= (uint32_t)(a.nm * a.nn))  // below 2^31
                return false;
            const uint32_t per = kBand * a.nn;
            const uint32_t b = a.nm <= kBand ? 0 : l / per, r = l - b * per;
            const uint32_t mc = min(kBand, a.nm - b * kBand);
            const uint32_t n = r / mc;
            t.kind = 0;
            t.m0 = (b * kBand + (r - n * mc)) * BM;
            t.n0 = n * kBN;
            t.k0 = 0;
            t.nk = a.nk;
            t.unit = n;
            t.piece = 0;
            return true;
        } else {
            for (; phase < a.pieces + a.lag; ++phase, stage = 0, j = 0) {
                if (stage == 0) {
                    if (phase < a.pieces) {
                        const int left = a.V - phase * a.Vc;
                        const uint32_t n_p = a.nm * (phase + 1 < a.pieces ? a.nn : (left + kBN - 1) / kBN);
                        const uint32_t r = turn(a, (uint32_t)phase * (uint32_t)(a.nm * a.nn));
                        if (r < n_p) {
                            const uint32_t n = r / (uint32_t)a.nm;
                            t.kind = 0;
                            t.m0 = (r - n * a.nm) * BM;
                            t.n0 = n * kBN;
                            t.k0 = 0;
                            t.nk = a.nk;
                            t.unit = 0;
                            t.piece = phase;
                            ++j;
                            return true;
                        }
                    }
                    stage = 1;
                    j = 0;
                }
                const int q = phase - a.lag;
                if (q < 0)
                    continue;
                const int vc = min(a.Vc, a.V - q * a.Vc);
                t.piece = q;
                if (stage == 1) {
                    const int kb = (vc + 63) / 64;
                    for (uint32_t u = c + j * a.C; u < (uint32_t)a.dh_units; u += a.C) {
                        ++j;
                        const uint32_t s = u / (uint32_t)a.dh_tiles, x = u - s * a.dh_tiles;
                        const uint32_t m = x / (uint32_t)a.nh;
                        t.k0 = (int)(s * kb / (uint32_t)a.dh_split);  // below 64 x 2^24
                        t.nk = (int)((s + 1) * kb / (uint32_t)a.dh_split) - t.k0;
                        if (t.nk == 0)  // a short last piece
                            continue;
                        t.kind = 1;
                        t.m0 = m * BM;
                        t.n0 = (x - m * a.nh) * kBN;
                        t.unit = u;
                        return true;
                    }
                    stage = 2;
                    j = 0;
                }
                if (!a.dw)
                    continue;
                const uint32_t tiles = (vc + BM - 1) / BM * a.nh, hi = (uint32_t)a.dh_units % a.C;
                const uint32_t first = min(tiles, a.dw_more * (a.C - hi));
                uint32_t l;
                if (stage == 2) {
                    l = j * (a.C - hi) + (c - hi);
                    if (j < (uint32_t)a.dw_more && c >= hi && l < first) {
                        ++j;
                    } else {
                        stage = 3;
                        j = 0;
                    }
                }
                if (stage == 3) {
                    const uint32_t all = (a.Vc + BM - 1) / BM * a.nh;
                    l = first + turn(a, (uint32_t)q * (all - min(all, a.dw_more * (a.C - hi))));
                    if (l >= tiles)
                        continue;
                    ++j;
                }
                const uint32_t m = l / (uint32_t)a.nh;
                t.kind = 2;
                t.m0 = m * BM;
                t.n0 = (l - m * a.nh) * kBN;
                t.k0 = 0;
                t.nk = a.dw_nk;
                t.unit = 0;
                return true;
            }
            return false;
        }
    }
};

constexpr int kTiles = 4;  // tiles known ahead

struct CeCtl {
    uint64_t full[6], empty[6], tfull[2], tempty[2];
    uint64_t tile_full[kTiles], tile_empty[kTiles], stored[kTiles];
    Tile tiles[kTiles];
    uint32_t tmem;
    int abort_flag;
};

// The tiles as one warp works them out (several divisions each) for the others,
// which only read them: done by each warp for itself, the thread that issues
// the MMAs would leave the tensor cores waiting between tiles (a fifth of the
// time of the backward pass at 4096 x 2048 x 32000).
struct Tiles {
    Ring r;

    // by the lanes in `mask` of a warp; false at the end, or where a wait gave up
    __device__ __forceinline__ bool next(CeCtl &c, Tile &t, uint32_t mask, volatile int *abort_flag, int32_t *status)
    {
        if (!__all_sync(mask, mbar_wait(smem_u32(&c.tile_full[r.i]), r.ph, abort_flag, status)))
            return false;
        t = c.tiles[r.i];
        __syncwarp(mask);
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(smem_u32(&c.tile_empty[r.i]));
        r.next(kTiles);
        return t.kind >= 0;
    }
};

// Bounded wait for a counter that other CTAs of the launch add to, before TMA
// copies of what they wrote (or over what they read).
__device__ __forceinline__ bool wait_count(const uint32_t *p, uint32_t want, volatile int *abort_flag,
                                           int32_t *status)
{
    const uint64_t t0 = global_ns();
    for (uint32_t n = 1;; ++n) {
        uint32_t v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        if (v >= want)
            break;
        if (*abort_flag)
            return false;
        if ((n & 15u) == 0 && global_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            if (status)
                sg_flag(status, SG_ERR_TIMEOUT);
            return false;
        }
        __nanosleep(64);
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    return true;
}

// One more.  PUBLISH: all writes that this thread knows of come before it (they
// have to be seen everywhere first, which takes a microsecond or two).
template <bool PUBLISH>
__device__ __forceinline__ void add_count(uint32_t *p)
{
    if constexpr (PUBLISH)
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
    else
        asm volatile("red.relaxed.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}

// Descriptors of an operand's tile at shared address `base`: the low word, to
// which stages (bytes / 16) and K steps are added, the high word, and the step.
// K-major: rows of 128 bytes of K, 8 rows to a swizzle atom.  MN-major: boxes
// of 64 rows (128 bytes) by 64 K, kBox apart.  Worked out once for a tile: the
// thread that issues the MMAs has little time for each.
struct OpDesc {
    uint32_t lo, hi, step;

    __device__ __forceinline__ OpDesc(uint32_t base, bool mn)
    {
        const uint64_t d = sdesc(base, mn ? kBox : 16, 1024, kLayoutSW128);
        lo = (uint32_t)d;
        hi = (uint32_t)(d >> 32);
        step = mn ? 2048 / 16 : 32 / 16;
    }
    __device__ __forceinline__ uint64_t at(uint32_t stage, int ks) const
    {
        return (uint64_t)hi << 32 | (lo + stage + ks * step);
    }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool f16)
{
    return f16 ? pack2_f16(a, b) : pack2(a, b);
}

// Factor of g before it is rounded to 16 bits; the products' epilogues take it
// out again.  It brings the largest |dloss| (1 - e), the target's part of g, to
// just `full` (1, or 2^14 in fp16, whose range would not hold dloss = 1 / T
// times a probability).  With the same dloss in every row, as in a mean, all
// targets' parts are then a little below a power of two, where a rounding is
// smallest against its value; without it they would all be rounded the same
// way at wherever 1 / T falls (measured at T = 777, fp16, e = 0.1: 4.3e-4 of
// error in dh instead of 2.7e-4 by the output's own rounding).  The epilogue
// warps of every CTA work it out while the first tile is under way.
__device__ __forceinline__ float g_scale(const CeArgs &a, float *sm)
{
    float top = 0.f;
    for (int t = threadIdx.x; t < a.T; t += kEpiWarps * 32) {
        const float v = fabsf(a.dloss[t]);
        if (v < INFINITY)
            top = fmaxf(top, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0)
        sm[threadIdx.x / 32] = top;
    named_bar(1, kEpiWarps * 32);
    for (int w = 0; w < kEpiWarps; ++w)
        top = fmaxf(top, sm[w]);
    // |g| <= |dloss|: with a factor of at least 1/2, g stays below 2 full
    top *= fmaxf(1.f - a.smooth, 0.5f);
    const bool plain = !(top >= 1e-30f && top <= 1e30f);
    const float s = plain ? 1.f : a.full / top;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.gscale[0] = s;
        a.gscale[1] = plain ? 1.f : top / a.full;
    }
    return s;
}

template <int CG, int MODE, bool F8>
__global__ void __launch_bounds__(kCeThreads, 1)
    k_ce(const __grid_constant__ CUtensorMap m_h, const __grid_constant__ CUtensorMap m_W,
         const __grid_constant__ CUtensorMap m_g, const CeArgs a)
{
    using K = Cfg<CG>;
    constexpr int NS = K::NS;
    constexpr int KE = F8 ? 128 : 64;  // elements of a K block
    __shared__ CeCtl c;
    __shared__ float sm_top[kEpiWarps];
    extern __shared__ uint8_t dsm[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int rank = CG == 2 ? (int)cluster_rank() : 0;
    const int cl = (int)blockIdx.x / CG;
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    if (threadIdx.x == 0) {
        c.abort_flag = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&c.full[s]), 1);
            mbar_init(smem_u32(&c.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&c.tfull[b]), 1);
            mbar_init(smem_u32(&c.tempty[b]), CG * kEpiWarps);
        }
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(smem_u32(&c.tile_full[i]), 1);
            mbar_init(smem_u32(&c.tile_empty[i]), kEpiWarps + 1 + (rank == 0) + (MODE == kBwd));
            mbar_init(smem_u32(&c.stored[i]), kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == kEpiWarps + 1) {
        tmem_alloc_cg<CG>(smem_u32(&c.tmem), 512);
        tmem_relinquish_cg<CG>();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2)
        cluster_sync();
    tc_fence_after();
    grid_wait();
    grid_go();
    const uint32_t tbase = c.tmem;
    volatile int *abort_flag = &c.abort_flag;
    Tile t;

    if (warp == kEpiWarps) {
        // ---------------------------------------------------------- producer
        if (lane == 0) {
            Ring r;
            bool ok = true;
            int seen = -1;  // last piece whose g was waited for
            for (Tiles tiles; ok && tiles.next(c, t, 1u, abort_flag, a.status);) {
                const bool a_mn = t.kind == 2, b_mn = t.kind != 0;
                const CUtensorMap *ma = t.kind ? &m_g : &m_h, *mb = t.kind == 2 ? &m_h : &m_W;
                // columns of g start at the piece's place, rows of W at the piece
                const int g_col = MODE == kBwd && t.kind ? t.piece % a.ring * a.Vc : 0;
                const int b_row = MODE == kBwd && t.kind != 2 ? t.piece * a.Vc : 0;
                const int am = t.m0 + rank * 128 + (a_mn ? g_col : 0), bn = t.n0 + rank * 128;
                if (MODE == kBwd && t.kind && t.piece != seen) {
                    const int left = min(a.Vc, a.V - t.piece * a.Vc);
                    seen = t.piece;
                    ok = wait_count(a.g_done + seen, (uint32_t)(a.nm * ((left + kBN - 1) / kBN)) * CG,
                                    abort_flag, a.status);
                    if (!ok)
                        break;
                }
                for (int kb = 0; kb < t.nk; ++kb) {
                    if (!mbar_wait(smem_u32(&c.empty[r.i]), r.ph ^ 1u, abort_flag, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = base + (uint32_t)r.i * K::kStage;
                    uint32_t bar = smem_u32(&c.full[r.i]);
                    if (rank == 0)
                        mbar_arrive_expect_tx(bar, CG * K::kStage);
                    if constexpr (CG == 2)
                        bar = mapa(bar, 0);
                    const int k = (t.k0 + kb) * KE;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        tma_load_2d_cg<CG>(st + j * kBox, ma, a_mn ? am + 64 * j : g_col + k, a_mn ? k : am + 64 * j,
                                           bar);
#pragma unroll
                    for (int j = 0; j < K::BRows / 64; ++j)
                        tma_load_2d_cg<CG>(st + K::kA + j * kBox, mb, b_mn ? bn + 64 * j : k,
                                           b_mn ? b_row + k : b_row + bn + 64 * j, bar);
                    r.next(NS);
                }
            }
            if (!ok) {
                // gave up: copies may still be on their way into this CTA (and
                // signal the pair's first CTA); they land long before this
                const uint64_t t0 = global_ns();
                while (global_ns() - t0 < 1000000u) {
                }
            }
        }
        __syncwarp();
    } else if (warp == kEpiWarps + 1) {
        // ---------------------------------------------------------- MMA
        if (rank == 0) {
            Ring r;
            int it = 0;
            bool ok = true;
            for (Tiles tiles; ok && tiles.next(c, t, 0xffffffffu, abort_flag, a.status);) {
                const bool a_mn = t.kind == 2, b_mn = t.kind != 0;
                const uint32_t idesc = (F8 || a.f16 ? idesc_f16(K::BM, kBN, a_mn, b_mn)
                                                    : idesc_bf16(K::BM, kBN, a_mn, b_mn));
                const OpDesc da(base, a_mn), db(base + K::kA, b_mn);
                const int buf = it & 1;
                ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&c.tempty[buf]),
                                                               ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, a.status));
                if (!ok)
                    break;
                tc_fence_after();
                for (int kb = 0; kb < t.nk; ++kb) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_cluster(smem_u32(&c.full[r.i]), r.ph, abort_flag, a.status));
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t st = (uint32_t)r.i * (K::kStage / 16);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_cg<CG, F8>(tbase + buf * kBN, da.at(st, ks), db.at(st, ks), idesc,
                                           (kb > 0 || ks > 0) ? 1u : 0u);
                        mma_commit_cg<CG>(smem_u32(&c.empty[r.i]));
                    }
                    __syncwarp();
                    r.next(NS);
                }
                if (ok && lane == 0)
                    mma_commit_cg<CG>(smem_u32(&c.tfull[buf]));
                __syncwarp();
                ++it;
            }
        }
    } else if (warp == kEpiWarps + 2) {
        // ---------------------------------------------------------- tiles
        if (lane == 0) {
            Ring r;
            Walk<CG, MODE> walk(cl);
            for (bool more = true; more; r.next(kTiles)) {
                more = walk.next(a, t);
                if (!more)
                    t.kind = -1;
                if (!mbar_wait(smem_u32(&c.tile_empty[r.i]), r.ph ^ 1u, abort_flag, a.status))
                    break;
                c.tiles[r.i] = t;
                mbar_arrive(smem_u32(&c.tile_full[r.i]));
            }
        }
        __syncwarp();
    } else if (warp == kEpiWarps + 3) {
        // ---------------------------------------------------------- signals
        // tells the other CTAs of each tile of g that the epilogue warps have
        // stored
        if (MODE == kBwd && lane == 0) {
            Ring r;
            uint32_t ph = 0;  // phase of stored, a bit for each place
            while (mbar_wait(smem_u32(&c.tile_full[r.i]), r.ph, abort_flag, a.status)) {
                t = c.tiles[r.i];
                if (t.kind < 0)
                    break;
                if (t.kind == 0) {
                    if (!mbar_wait(smem_u32(&c.stored[r.i]), (ph >> r.i) & 1u, abort_flag, a.status))
                        break;
                    ph ^= 1u << r.i;
                    add_count<true>(a.g_done + t.piece);
                }
                mbar_arrive(smem_u32(&c.tile_empty[r.i]));
                r.next(kTiles);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- epilogue
        // a warp reads its quarter of the TMEM lanes (tile rows) and one half
        // of the tile's columns; a thread has one row
        const int q = warp & 3, half = warp >> 2;
        const int row_in = rank * 128 + q * 32 + lane;
        [[maybe_unused]] uint32_t *stg =
            reinterpret_cast<uint32_t *>(dsm + (base - smem_u32(dsm)) + NS * K::kStage + warp * kStgWarp);
        float m2 = -INFINITY, s = 0.f, zs = 0.f;
        [[maybe_unused]] float scale = 1.f, inv = 1.f;
        [[maybe_unused]] int freed = a.ring - 1;  // g of pieces up to this may be written
        if constexpr (MODE == kBwd) {
            scale = g_scale(a, sm_top);
            inv = 1.f / scale;
        }
        int it = 0;
        Tiles tiles;
        for (;;) {
            [[maybe_unused]] const int slot = tiles.r.i;
            if (!tiles.next(c, t, 0xffffffffu, abort_flag, a.status))
                break;
            const int buf = it & 1;
            const int row = t.m0 + row_in;              // row of the tile's A operand
            const int col0 = t.n0 + half * (kBN / 2);   // first column of this warp
            const int v0 = MODE == kBwd ? t.piece * a.Vc : 0;
            const uint32_t tm = tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kBN + half * (kBN / 2));
            // what the row needs, before the wait
            int tgt = -1;
            [[maybe_unused]] float cf = 0.f, l2 = 0.f, hs = 1.f;
            if (MODE == kLse || t.kind == 0) {
                if (row < a.T) {
                    const int y = a.targets[row];
                    const bool live = y != a.ignore && y >= 0 && y < a.V;
                    if (live)
                        tgt = y - v0 - col0;  // this warp's column of the target, if it has it
                    if constexpr (MODE == kBwd) {
                        l2 = a.lse[row] * kLog2e;
                        if (live)
                            cf = a.dloss[row] * scale;
                    } else if constexpr (F8) {
                        hs = a.h_scale ? a.h_scale[row] : 1.f;
                    }
                }
                if (MODE == kBwd && t.piece > freed) {
                    // the place of this piece's g was another's
                    bool ok = true;
                    if (lane == 0)
                        ok = wait_count(a.w_done + t.piece - a.ring, (uint32_t)(a.dh_units + (a.dw ? (a.Vc + K::BM - 1) / K::BM * a.nh : 0)),
                                        abort_flag, a.status);
                    if (!__all_sync(0xffffffffu, ok))
                        break;
                    freed = t.piece;
                }
            }
            if (!__all_sync(0xffffffffu,
                            mbar_wait_cluster(smem_u32(&c.tfull[buf]), (uint32_t)(it >> 1) & 1u, abort_flag, a.status)))
                break;
            tc_fence_after();
            // all of a gradient tile's operands have been read
            if (MODE == kBwd && t.kind && threadIdx.x == 0 && rank == 0)
                add_count<false>(a.w_done + t.piece);
            if constexpr (MODE == kLse) {
                const int left = a.V - col0;  // columns of the vocabulary from col0 on
#pragma unroll 1
                for (int cc = 0; cc < kBN / 2; cc += 32) {
                    float v[32];
                    tmem_ld_chunk<32>(tm + cc, v);
                    if constexpr (F8) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[x] *= hs * (a.W_scale && cc + x < left ? __ldg(a.W_scale + col0 + cc + x) : 1.f);
                    }
                    if (tgt >= cc && tgt < cc + 32) {
                        // in this form so that v stays in registers (an index
                        // known only at run time would put it into memory,
                        // for every chunk)
                        float z = 0.f;
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            asm("{\n\t.reg .pred p;\n\t"
                                "setp.eq.s32 p, %2, %3;\n\t"
                                "@p mov.f32 %0, %1;\n\t}"
                                : "+f"(z)
                                : "f"(v[x]), "r"(tgt - cc), "r"(x));
                        a.ztgt[row] = z;
                    }
                    if (a.zsum) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            zs += cc + x < left ? v[x] : 0.f;
                    }
                    if (cc + 32 > left) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (cc + x >= left)
                                v[x] = -INFINITY;
                    }
                    float top = v[0];
#pragma unroll
                    for (int x = 1; x < 32; ++x)
                        top = fmaxf(top, v[x]);
                    const float m = fmaxf(m2, top * kLog2e);
                    const float mm = m == -INFINITY ? 0.f : m;
                    float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        p[x & 3] += ex2(fmaf(v[x], kLog2e, -mm));
                    s = fmaf(s, ex2(m2 - mm), (p[0] + p[1]) + (p[2] + p[3]));
                    m2 = m;
                }
                // one row tile: the running values cover all tiles of this
                // CTA; else they are written out for every tile
                if (a.nm > 1) {
                    const int64_t at = (int64_t)(t.unit * 2 + half) * a.Tp + row;
                    a.part[at] = make_float2(m2, s);
                    if (a.zsum)
                        a.zsum[at] = zs;
                    m2 = -INFINITY;
                    s = zs = 0.f;
                }
            } else if (t.kind == 0) {
                const int left = a.V - v0 - col0;
                const int g_col = t.piece % a.ring * a.Vc + col0;
                const float off = cf * (a.smooth / (float)a.V), hit = cf * (1.f - a.smooth);
#pragma unroll 1
                for (int cc = 0; cc < kBN / 2; cc += 32) {
                    float v[32];
                    tmem_ld_chunk<32>(tm + cc, v);
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        v[x] = cf == 0.f ? 0.f : fmaf(ex2(fmaf(v[x], kLog2e, -l2)), cf, -off);
                    if (tgt >= cc && tgt < cc + 32) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[x] -= x == tgt - cc ? hit : 0.f;
                    }
                    if (cc + 32 > left) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (cc + x >= left)
                                v[x] = 0.f;
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        w[x] = pack16(v[2 * x], v[2 * x + 1], a.f16);
                    if (row < a.T) {
                        uint16_t *dst = a.g + (int64_t)row * a.ldg + g_col + cc;
                        st_global32(dst, w);
                        st_global32(dst + 16, w + 8);
                    }
                }
            } else {
                if (t.kind == 1) {
                    // always this thread's own sums, one piece after the other
                    float4 *acc = reinterpret_cast<float4 *>(a.acc) +
                                  ((int64_t)(t.unit * CG + rank) * (kBN / 4) + half * (kBN / 8)) * 128 + q * 32 + lane;
#pragma unroll 1
                    for (int cc = 0; cc < kBN / 2; cc += 32) {
                        float v[32];
                        tmem_ld_chunk<32>(tm + cc, v);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            float4 *p = acc + (cc / 4 + x) * 128;
                            if (t.piece == 0)
                                *p = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                            else
                                red_add_v4(&p->x, v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                        }
                    }
                } else {
                    const int64_t row0 = (int64_t)v0 + t.m0 + rank * 128 + q * 32;  // the warp's first row of dW
#pragma unroll 1
                    for (int cc = 0; cc < kBN / 2; cc += 32) {
                        float v[32];
                        tmem_ld_chunk<32>(tm + cc, v);
                        uint32_t w[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            w[x] = pack16(v[2 * x] * inv, v[2 * x + 1] * inv, a.f16);
                        const int x0 = col0 + cc;
                        if (a.dw_align == 32) {
                            if (row0 + lane < a.V) {
                                uint16_t *dst = a.dW + (row0 + lane) * a.lddW + x0;
                                if (x0 < a.H)
                                    st_global32(dst, w);
                                if (x0 + 16 < a.H)
                                    st_global32(dst + 16, w + 8);
                            }
                        } else if (a.dw_align == 16) {
                            if (row0 + lane < a.V) {
                                uint16_t *dst = a.dW + (row0 + lane) * a.lddW + x0;
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    if (x0 + 8 * x < a.H)
                                        *reinterpret_cast<uint4 *>(dst + 8 * x) =
                                            make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                            }
                        } else {
                            // rows on any boundary: through shared memory, so
                            // that a warp writes a row at a time
                            __syncwarp();
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                stg[lane * 17 + x] = w[x];
                            __syncwarp();
                            for (int r = 0; r < 32 && row0 + r < a.V; ++r)
                                if (x0 + lane < a.H)
                                    a.dW[(row0 + r) * a.lddW + x0 + lane] =
                                        reinterpret_cast<const uint16_t *>(stg + r * 17)[lane];
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = smem_u32(&c.tempty[buf]);
                // the accumulator's values are in registers already (wait::ld):
                // nothing in memory has to be visible with this arrival
                if constexpr (CG == 2)
                    mbar_arrive_remote_relaxed(mapa(bar, 0));
                else
                    mbar_arrive(bar);
                if (MODE == kBwd && t.kind == 0)
                    mbar_arrive(smem_u32(&c.stored[slot]));
            }
            __syncwarp();
            ++it;
        }
        if constexpr (MODE == kLse) {
            if (a.nm == 1) {
                const int64_t at = (int64_t)row_in * (2 * a.C) + cl * 2 + half;
                a.part[at] = make_float2(m2, s);
                if (a.zsum)
                    a.zsum[at] = zs;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2)
        cluster_sync();
    if (warp == kEpiWarps + 1) {
        tc_fence_after();
        tmem_dealloc_cg<CG>(tbase, 512);
    }
}

// ---------------------------------------------------------------- small kernels
// one more partial maximum (of z log2 e) and sum
__device__ __forceinline__ void join_one(float &m, float &s, float2 p)
{
    const float mn = fmaxf(m, p.x), ms = mn == -INFINITY ? 0.f : mn;
    s = s * exp2f(m - ms) + p.y * exp2f(p.x - ms);
    m = mn;
}

struct JoinArgs {
    const float2 *part;
    const float *zsum, *ztgt;
    const int32_t *targets;
    float *loss, *lse;
    int32_t *status;
    int32_t slots, Tp, T, V, ignore;
    float smooth;
};

__device__ __forceinline__ void join_out(const JoinArgs &a, int t, float m, float s, float zs)
{
    const float l = (m + log2f(s)) * kLn2;
    a.lse[t] = l;
    const int y = a.targets[t];
    float out = 0.f;
    if (y >= 0 && y < a.V && y != a.ignore) {
        out = l - (1.f - a.smooth) * a.ztgt[t];
        if (a.zsum)
            out -= a.smooth * (zs / (float)a.V);
    } else if (y != a.ignore && a.status) {
        sg_flag(a.status, SG_ERR_DATA);
    }
    a.loss[t] = out;
}

// lse and loss of 32 rows from their partial maxima and sums, [slot][row]
__global__ void __launch_bounds__(1024) k_ce_join(const JoinArgs a)
{
    __shared__ float2 sm[32][33];
    __shared__ float sz[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int t = blockIdx.x * 32 + lane;  // below Tp, a multiple of 128
    float m = -INFINITY, s = 0.f, zs = 0.f;
    grid_wait();
    for (int i = warp; i < a.slots; i += 32) {
        join_one(m, s, a.part[(int64_t)i * a.Tp + t]);
        if (a.zsum)
            zs += a.zsum[(int64_t)i * a.Tp + t];
    }
    sm[warp][lane] = make_float2(m, s);
    sz[warp][lane] = zs;
    __syncthreads();
    if (warp != 0 || t >= a.T)
        return;
    for (int w = 1; w < 32; ++w) {
        join_one(m, s, sm[w][lane]);
        zs += sz[w][lane];
    }
    join_out(a, t, m, s, zs);
}

// the same for one row tile, [row][slot]: a CTA for a row, whose slots (at most
// 3 x 128) are loaded together
__global__ void __launch_bounds__(128) k_ce_join_row(const JoinArgs a)
{
    __shared__ float sm[3][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, t = blockIdx.x;
    float2 p[3];
    float zs = 0.f;
    grid_wait();
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int i = threadIdx.x + 128 * j;
        const bool in = i < a.slots;
        p[j] = in ? a.part[(int64_t)t * a.slots + i] : make_float2(-INFINITY, 0.f);
        if (a.zsum)
            zs += in ? a.zsum[(int64_t)t * a.slots + i] : 0.f;
    }
    float m = fmaxf(fmaxf(p[0].x, p[1].x), p[2].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0)
        sm[0][warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sm[0][0], sm[0][1]), fmaxf(sm[0][2], sm[0][3]));
    const float ms = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        s += p[j].y * exp2f(p[j].x - ms);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        zs += __shfl_xor_sync(0xffffffffu, zs, o);
    }
    if (lane == 0) {
        sm[1][warp] = s;
        sm[2][warp] = zs;
    }
    __syncthreads();
    if (threadIdx.x == 0)
        join_out(a, t, m, (sm[1][0] + sm[1][1]) + (sm[1][2] + sm[1][3]),
                 (sm[2][0] + sm[2][1]) + (sm[2][2] + sm[2][3]));
}

// dh = the sum of its pieces, 32 rows x 32 columns to a CTA, a warp for four
// columns
template <int CG>
__global__ void __launch_bounds__(256)
    k_ce_dh(const float4 *__restrict__ acc, int tiles, int nn, int split, int T, int H,
            const float *__restrict__ gscale, int f16, uint16_t *__restrict__ dh, int64_t lddh)
{
    __shared__ uint16_t sm[32][34];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int x = blockIdx.x / (CG * 4), rq = blockIdx.x % (CG * 4);  // tile, 32-row part of it
    const int row0 = x / nn * Cfg<CG>::BM + rq * 32, col0 = x % nn * kBN + blockIdx.y * 32;
    if (row0 >= T || col0 >= H)
        return;
    grid_wait();
    const float inv = gscale[1];
    const float4 *src =
        acc + (((int64_t)x * CG + rq / 4) * (kBN / 4) + blockIdx.y * 8 + warp) * 128 + (rq & 3) * 32 + lane;
    const int64_t step = (int64_t)tiles * CG * (kBN / 4) * 128;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < split; ++s) {
        const float4 o = src[s * step];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
    }
    *reinterpret_cast<uint32_t *>(&sm[lane][warp * 4]) = pack16(v.x * inv, v.y * inv, f16);
    *reinterpret_cast<uint32_t *>(&sm[lane][warp * 4 + 2]) = pack16(v.z * inv, v.w * inv, f16);
    __syncthreads();
    for (int r = warp; r < 32 && row0 + r < T; r += 8)
        if (col0 + lane < H)
            dh[(int64_t)(row0 + r) * lddh + col0 + lane] = sm[r][lane];
}

// rows that do not start on 16 bytes, copied to a stride that does
template <typename E>
__global__ void __launch_bounds__(256)
    k_ce_pack(const E *__restrict__ src, int64_t ld, int64_t rows, int cols, E *__restrict__ dst, int64_t ldd)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += 256)
            dst[r * ldd + c] = src[r * ld + c];
}

// ---------------------------------------------------------------- host
std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode_ce{nullptr};

// row-major matrix in boxes of 64 rows x 128 bytes, 128-byte swizzle
sg_status map_of(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t ld, int elem,
                 const char *what)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = g_encode_ce.load(std::memory_order_acquire);
    if (!enc) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn) {
            cudaGetLastError();
            CE_FAIL(SG_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
        }
        enc = (PFN_cuTensorMapEncodeTiled_v12000)fn;
        g_encode_ce.store(enc, std::memory_order_release);
    }
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld * elem)};
    cuuint32_t box[2] = {128u / (uint32_t)elem, 64u};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                           const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        CE_FAIL(SG_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", what, (int)r);
    return SG_OK;
}

// `after`: the kernel before it in the stream is one of this call's, which this
// one may overlap; `together`: its CTAs wait for one another
template <typename... P, typename... A>
sg_status launch(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster, bool after,
                 bool together, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[3];
    cfg.attrs = at;
    cfg.numAttrs = 0;
    if (cluster > 1) {
        at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
        at[cfg.numAttrs].val.clusterDim.y = 1;
        at[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    if (after) {
        at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (together) {
        at[cfg.numAttrs].id = cudaLaunchAttributeCooperative;
        at[cfg.numAttrs++].val.cooperative = 1;
    }
    SG_TRY_CUDA(cudaLaunchKernelEx(&cfg, kernel, args...));
    return SG_OK;
}

// clusters of CG CTAs that run at the same time (the backward kernel's wait for
// one another), and the kernel made ready for the current device
template <int CG, int MODE, bool F8>
sg_status prepare_ce(int *clusters)
{
    static std::atomic<int> known[64];  // by device
    int dev = 0;
    SG_TRY_CUDA(cudaGetDevice(&dev));
    int n = known[dev & 63].load(std::memory_order_acquire);
    if (n == 0) {
        SG_TRY_CUDA(cudaFuncSetAttribute(k_ce<CG, MODE, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Cfg<CG>::kSmem));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kSMs / CG * CG);
        cfg.blockDim = dim3(kCeThreads);
        cfg.dynamicSmemBytes = Cfg<CG>::kSmem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = CG;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        SG_TRY_CUDA(cudaOccupancyMaxActiveClusters(&n, k_ce<CG, MODE, F8>, &cfg));
        if (n < 1)
            CE_FAIL(SG_ERR_CUDA, "no cluster of %d CTAs of the softmax kernel fits this device", CG);
        if (n > kSMs / CG)
            n = kSMs / CG;
        known[dev & 63].store(n, std::memory_order_release);
    }
    *clusters = n;
    return SG_OK;
}

template <int CG, int MODE, bool F8>
sg_status launch_ce(const CUtensorMap &h, const CUtensorMap &W, const CUtensorMap &g, const CeArgs &a,
                    cudaStream_t st)
{
    return launch(k_ce<CG, MODE, F8>, dim3((unsigned)a.C * CG), kCeThreads, (int)Cfg<CG>::kSmem, CG, false,
                  MODE == kBwd, st, h, W, g, a);
}

// One call's tiles and the places of its work memory
struct Plan {
    int es = 2, CG = 1, BM = 128, C = 1;
    bool pack_h = false, pack_W = false;
    int64_t ldp = 0;             // row stride of the packed copies
    int64_t nm = 0, Tp = 0;
    // forward
    int64_t slots = 0;
    // backward
    int64_t Vc = 0, pieces = 0, lag = 0, ring = 0;
    int64_t dh_nn = 0, dh_tiles = 0, split = 1, dw_more = 0;
    // byte offsets
    int64_t o_h = 0, o_W = 0, o_part = 0, o_zsum = 0, o_ztgt = 0, o_count = 0, o_gs = 0, o_g = 0, o_acc = 0, bytes = 0;
};

bool tma_ok(const void *p, int64_t ld, int64_t es) { return ((uintptr_t)p & 15) == 0 && (ld * es) % 16 == 0; }

// Time of a tile or dh unit of nk K blocks, in half K blocks: a tile that is
// shorter than its output takes to reach memory (2 K blocks of a CTA, 4 of a
// pair) costs that, and each has a little of its own.
int64_t tile_cost(int64_t nk, int CG) { return 2 * (nk > 2 * CG ? nk : 2 * CG) + 1; }

sg_status make_plan(const void *h, int64_t ldh, int64_t T, int64_t H, const void *W, int64_t ldw, int64_t V,
                    int32_t dtype, bool backward, Plan *p)
{
    p->es = dtype == SG_E4M3 ? 1 : 2;
    p->CG = T > 128 ? 2 : 1;
    p->BM = 128 * p->CG;
    if (backward)
        CE_TRY(p->CG == 1 ? (prepare_ce<1, kBwd, false>(&p->C)) : (prepare_ce<2, kBwd, false>(&p->C)));
    else if (dtype == SG_E4M3)
        CE_TRY(p->CG == 1 ? (prepare_ce<1, kLse, true>(&p->C)) : (prepare_ce<2, kLse, true>(&p->C)));
    else
        CE_TRY(p->CG == 1 ? (prepare_ce<1, kLse, false>(&p->C)) : (prepare_ce<2, kLse, false>(&p->C)));
    p->pack_h = !tma_ok(h, ldh, p->es);
    p->pack_W = !tma_ok(W, ldw, p->es);
    p->ldp = ceil_div(H * p->es, 16) * 16 / p->es;
    p->nm = ceil_div(T, p->BM);
    p->Tp = p->nm * p->BM;
    auto take = [&](int64_t n) {
        const int64_t at = p->bytes;
        p->bytes += ceil_div(n, 256) * 256;
        return at;
    };
    if (p->pack_h)
        p->o_h = take(T * p->ldp * p->es);
    if (p->pack_W)
        p->o_W = take(V * p->ldp * p->es);
    if (!backward) {
        p->slots = 2 * (p->nm == 1 ? (int64_t)p->C : ceil_div(V, kBN));
        p->o_part = take(p->slots * p->Tp * 8);
        p->o_zsum = take(p->slots * p->Tp * 4);
        p->o_ztgt = take(T * 4);
        return SG_OK;
    }
    int64_t Vc = (getenv("SG_W") ? atoll(getenv("SG_W")) : (24ll << 20)) / (2 * H) / kBN * kBN;
    if (Vc < kBN)
        Vc = kBN;
    const int64_t most = (getenv("SG_G") ? atoll(getenv("SG_G")) : (64ll << 20)) / (2 * T) / kBN * kBN;
    if (Vc > most)
        Vc = most < kBN ? kBN : most;
    const int64_t all = ceil_div(V, kBN) * kBN;
    if (Vc > all)
        Vc = all;
    p->Vc = Vc;
    p->pieces = ceil_div(V, Vc);
    p->lag = getenv("SG_L") ? atoll(getenv("SG_L")) : 1;
    p->ring = p->lag + 2 < p->pieces ? p->lag + 2 : p->pieces;
    p->dh_nn = ceil_div(H, kBN);
    p->dh_tiles = p->nm * p->dh_nn;
    // split K of dh until its units leave room for the other tiles' even share
    const int64_t kb = ceil_div(V < Vc ? V : Vc, 64), nk = ceil_div(H, 64), tk = ceil_div(T, 64);
    const int64_t logit = p->nm * (Vc / kBN) * tile_cost(nk, p->CG);
    const int64_t dw = ceil_div(Vc, p->BM) * p->dh_nn * tile_cost(tk, p->CG);
    double best = 0;
    for (int64_t n = 1; n <= kb && n <= 64; ++n) {
        const int64_t units = p->dh_tiles * n, cost = tile_cost(ceil_div(kb, n), p->CG) + 2;
        const double even = (double)(units * cost + dw + logit) / p->C;
        const double last = (double)(ceil_div(units, p->C) * cost) + (double)logit / p->C;
        const double span = (even > last ? even : last) * (1.0 + 0.002 * (double)n);
        if (n == 1 || span < best) {
            best = span;
            p->split = n;
        }
    }
    p->dw_more = (tile_cost(ceil_div(kb, p->split), p->CG) + 2) / tile_cost(tk, p->CG);
    p->o_count = take(p->pieces * 8);
    p->o_gs = take(8);
    p->o_g = take(T * p->ring * Vc * 2);
    p->o_acc = take(p->dh_tiles * p->split * p->BM * kBN * 4);
    return SG_OK;
}

sg_status check_ce(const char *fn, const void *h, int64_t ldh, int64_t T, int64_t H, const void *W, int64_t ldw,
                   int64_t V, int32_t dtype, bool backward)
{
    if (dtype != SG_BF16 && dtype != SG_F16 && (dtype != SG_E4M3 || backward))
        CE_FAIL(SG_ERR_INVALID, "%s: dtype %d is not SG_BF16 or SG_F16%s", fn, dtype,
                backward ? "" : " or SG_E4M3");
    if (T < 0 || H < 1 || V < 1)
        CE_FAIL(SG_ERR_INVALID, "%s: need T >= 0, H >= 1 and V >= 1 (T=%lld H=%lld V=%lld)", fn, (long long)T,
                (long long)H, (long long)V);
    // the last: tiles are counted in 31 bits
    if (T > (1 << 24) || H > (1 << 20) || V > (1ll << 30) || ceil_div(T, 128) * ceil_div(V, 128) >= (1ll << 31))
        CE_FAIL(SG_ERR_UNSUPPORTED, "%s: T=%lld, H=%lld, V=%lld or T V is above 2^24, 2^20, 2^30 or 2^45", fn,
                (long long)T, (long long)H, (long long)V);
    if (ldh < H || ldw < H)
        CE_FAIL(SG_ERR_INVALID, "%s: a row stride (%lld, %lld) is below H=%lld", fn, (long long)ldh, (long long)ldw,
                (long long)H);
    const int64_t es = dtype == SG_E4M3 ? 1 : 2;
    if ((uintptr_t)h % es != 0 || (uintptr_t)W % es != 0)
        CE_FAIL(SG_ERR_INVALID, "%s: h or W is not aligned to its elements", fn);
    return SG_OK;
}

template <typename E>
void pack(const void *src, int64_t ld, int64_t rows, int64_t cols, void *dst, int64_t ldd, cudaStream_t st)
{
    const int64_t grid = rows < 152 * 8 ? rows : 152 * 8;
    k_ce_pack<E><<<(unsigned)grid, 256, 0, st>>>(static_cast<const E *>(src), ld, rows, (int)cols,
                                                 static_cast<E *>(dst), ldd);
}

// maps of h and W, packed first where their rows need it
sg_status operand_maps(const Plan &p, const void *h, int64_t ldh, int64_t T, int64_t H, const void *W, int64_t ldw,
                       int64_t V, uint8_t *work, CUtensorMap *mh, CUtensorMap *mW, cudaStream_t st)
{
    auto packed = [&](const void *&src, int64_t &ld, int64_t rows, int64_t at) {
        if (p.es == 1)
            pack<uint8_t>(src, ld, rows, H, work + at, p.ldp, st);
        else
            pack<uint16_t>(src, ld, rows, H, work + at, p.ldp, st);
        src = work + at;
        ld = p.ldp;
    };
    if (p.pack_h)
        packed(h, ldh, T, p.o_h);
    if (p.pack_W)
        packed(W, ldw, V, p.o_W);
    SG_TRY_CUDA(cudaGetLastError());
    CE_TRY(map_of(mh, h, H, T, ldh, p.es, "h"));
    return map_of(mW, W, H, V, ldw, p.es, "W");
}

}  // namespace

extern "C" {

sg_status sg_softmax_ce_work(const void *h, int64_t ldh, int64_t T, int64_t H, const void *W, int64_t ldw, int64_t V,
                             int32_t dtype, int32_t backward, int64_t *bytes)
{
    const char *fn = "sg_softmax_ce_work";
    if (!bytes)
        CE_FAIL(SG_ERR_INVALID, "%s: bytes is NULL", fn);
    CE_TRY(check_ce(fn, h, ldh, T, H, W, ldw, V, dtype, backward != 0));
    Plan p;
    if (T > 0)
        CE_TRY(make_plan(h, ldh, T, H, W, ldw, V, dtype, backward != 0, &p));
    *bytes = p.bytes;
    return SG_OK;
}

sg_status sg_softmax_ce_fwd(const void *h, int64_t ldh, const float *h_scale, int64_t T, int64_t H, const void *W,
                            int64_t ldw, const float *W_scale, int64_t V, int32_t dtype, const int32_t *targets,
                            int32_t ignore_index, double smoothing, float *loss, float *lse, void *work,
                            int64_t work_bytes, int32_t *status, void *stream)
{
    const char *fn = "sg_softmax_ce_fwd";
    NvtxRange nvtx_(fn);
    CE_TRY(check_ce(fn, h, ldh, T, H, W, ldw, V, dtype, false));
    if (!W || (T && (!h || !targets || !loss || !lse)))
        CE_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL", fn);
    if ((h_scale || W_scale) && dtype != SG_E4M3)
        CE_FAIL(SG_ERR_INVALID, "%s: scales go with SG_E4M3 rows only", fn);
    if (!(smoothing >= 0.0 && smoothing <= 1.0))
        CE_FAIL(SG_ERR_INVALID, "%s: smoothing=%g is outside [0, 1]", fn, smoothing);
    if (T == 0)
        return SG_OK;
    Plan p;
    CE_TRY(make_plan(h, ldh, T, H, W, ldw, V, dtype, false, &p));
    if (!work || work_bytes < p.bytes || ((uintptr_t)work & 255) != 0)
        CE_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_softmax_ce_work), aligned to 256", fn,
                (long long)p.bytes);
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t *w8 = static_cast<uint8_t *>(work);
    CUtensorMap mh, mW;
    CE_TRY(operand_maps(p, h, ldh, T, H, W, ldw, V, w8, &mh, &mW, st));
    CeArgs a = {};
    a.T = (int32_t)T;
    a.V = (int32_t)V;
    a.H = (int32_t)H;
    a.C = p.C;
    a.nm = (int32_t)p.nm;
    a.nn = (int32_t)ceil_div(V, kBN);
    a.nk = (int32_t)ceil_div(H * p.es, 128);
    a.f16 = dtype == SG_F16;
    a.h_scale = h_scale;
    a.W_scale = W_scale;
    a.targets = targets;
    a.ignore = ignore_index;
    a.part = reinterpret_cast<float2 *>(w8 + p.o_part);
    a.zsum = smoothing > 0 ? reinterpret_cast<float *>(w8 + p.o_zsum) : nullptr;
    a.ztgt = reinterpret_cast<float *>(w8 + p.o_ztgt);
    a.Tp = (int32_t)p.Tp;
    a.status = status;
    if (dtype == SG_E4M3)
        CE_TRY(p.CG == 1 ? (launch_ce<1, kLse, true>(mh, mW, mh, a, st))
                         : (launch_ce<2, kLse, true>(mh, mW, mh, a, st)));
    else
        CE_TRY(p.CG == 1 ? (launch_ce<1, kLse, false>(mh, mW, mh, a, st))
                         : (launch_ce<2, kLse, false>(mh, mW, mh, a, st)));
    JoinArgs j;
    j.part = a.part, j.zsum = a.zsum, j.ztgt = a.ztgt, j.targets = targets, j.loss = loss, j.lse = lse;
    j.status = status, j.slots = (int32_t)p.slots, j.Tp = a.Tp, j.T = a.T, j.V = a.V, j.ignore = ignore_index;
    j.smooth = (float)smoothing;
    if (p.nm == 1)
        return launch(k_ce_join_row, dim3((unsigned)T), 128, 0, 1, true, false, st, j);
    return launch(k_ce_join, dim3((unsigned)ceil_div(T, 32)), 1024, 0, 1, true, false, st, j);
}

sg_status sg_softmax_ce_bwd(const void *h, int64_t ldh, int64_t T, int64_t H, const void *W, int64_t ldw, int64_t V,
                            int32_t dtype, const int32_t *targets, int32_t ignore_index, double smoothing,
                            const float *lse, const float *dloss, void *dh, int64_t lddh, void *dW, int64_t lddw,
                            void *work, int64_t work_bytes, int32_t *status, void *stream)
{
    const char *fn = "sg_softmax_ce_bwd";
    NvtxRange nvtx_(fn);
    CE_TRY(check_ce(fn, h, ldh, T, H, W, ldw, V, dtype, true));
    if (!W || (T && (!h || !targets || !lse || !dloss)) || (!dh && !dW))
        CE_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL", fn);
    if (!(smoothing >= 0.0 && smoothing <= 1.0))
        CE_FAIL(SG_ERR_INVALID, "%s: smoothing=%g is outside [0, 1]", fn, smoothing);
    if ((dh && (lddh < H || (uintptr_t)dh % 2 != 0)) || (dW && (lddw < H || (uintptr_t)dW % 2 != 0)))
        CE_FAIL(SG_ERR_INVALID, "%s: dh or dW has a row stride below H or is not aligned to its elements", fn);
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {
        if (dW)
            SG_TRY_CUDA(cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)H * 2, (size_t)V, st));
        return SG_OK;
    }
    Plan p;
    CE_TRY(make_plan(h, ldh, T, H, W, ldw, V, dtype, true, &p));
    if (!work || work_bytes < p.bytes || ((uintptr_t)work & 255) != 0)
        CE_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_softmax_ce_work), aligned to 256", fn,
                (long long)p.bytes);
    uint8_t *w8 = static_cast<uint8_t *>(work);
    CUtensorMap mh, mW, mg;
    CE_TRY(operand_maps(p, h, ldh, T, H, W, ldw, V, w8, &mh, &mW, st));
    CE_TRY(map_of(&mg, w8 + p.o_g, p.ring * p.Vc, T, p.ring * p.Vc, 2, "g"));
    CeArgs a = {};
    a.T = (int32_t)T;
    a.V = (int32_t)V;
    a.H = (int32_t)H;
    a.C = p.C;
    a.nm = (int32_t)p.nm;
    a.nn = (int32_t)(p.Vc / kBN);
    a.nk = (int32_t)ceil_div(H, 64);
    a.f16 = dtype == SG_F16;
    a.targets = targets;
    a.ignore = ignore_index;
    a.status = status;
    a.lse = lse;
    a.dloss = dloss;
    a.gscale = reinterpret_cast<float *>(w8 + p.o_gs);
    a.smooth = (float)smoothing;
    a.full = dtype == SG_F16 ? 16384.f : 1.f;
    a.pieces = (int32_t)p.pieces;
    a.Vc = (int32_t)p.Vc;
    a.lag = (int32_t)p.lag;
    a.ring = (int32_t)p.ring;
    a.nh = (int32_t)p.dh_nn;
    a.dh_tiles = (int32_t)p.dh_tiles;
    a.dh_split = (int32_t)p.split;
    a.dh_units = dh ? (int32_t)(p.dh_tiles * p.split) : 0;
    a.dw = dW != nullptr;
    a.dw_nk = (int32_t)ceil_div(T, 64);
    a.dw_more = dh ? (int32_t)p.dw_more : 0;
    a.acc = reinterpret_cast<float *>(w8 + p.o_acc);
    a.g = reinterpret_cast<uint16_t *>(w8 + p.o_g);
    a.ldg = p.ring * p.Vc;
    a.dW = static_cast<uint16_t *>(dW);
    a.lddW = lddw;
    const uintptr_t bits = (uintptr_t)dW | (uintptr_t)(lddw * 2) | (uintptr_t)(H * 2);
    a.dw_align = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 2;
    a.g_done = reinterpret_cast<uint32_t *>(w8 + p.o_count);
    a.w_done = a.g_done + p.pieces;
    SG_TRY_CUDA(cudaMemsetAsync(a.g_done, 0, (size_t)p.pieces * 8, st));
    CE_TRY(p.CG == 1 ? (launch_ce<1, kBwd, false>(mh, mW, mg, a, st))
                     : (launch_ce<2, kBwd, false>(mh, mW, mg, a, st)));
    if (dh) {
        const dim3 grid((unsigned)(p.dh_tiles * p.CG * 4), kBN / 32);
        const float4 *acc = reinterpret_cast<const float4 *>(a.acc);
        return launch(p.CG == 1 ? k_ce_dh<1> : k_ce_dh<2>, grid, 256, 0, 1, true, false, st, acc, (int)p.dh_tiles,
                      (int)p.dh_nn, (int)p.split, (int)T, (int)H, (const float *)a.gscale, (int)a.f16,
                      static_cast<uint16_t *>(dh), lddh);
    }
    return SG_OK;
}

}  // extern "C"
