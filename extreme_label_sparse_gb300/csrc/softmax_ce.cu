// Softmax cross entropy over a large label set (definitions in include/sg.h):
//   z = h W^T,  lse_t = log sum_v exp z_tv,
//   loss_t = lse_t - (1 - e) z_t,y - e mean_v z_t,
//   g_tv = dloss_t (exp(z_tv - lse_t) - (1 - e) [v = y_t] - e / V),
//   dh = g W,  dW = g^T h.
// The logits never reach memory.  Forward: one matrix product whose epilogue
// reduces each tile of logits to a running maximum and sum per row; a small
// kernel joins them.  (Where those would take more than 256 MB, bands of rows
// and pieces of the vocabulary in turn.)  Backward, over pieces of the vocabulary: the product
// again, its epilogue turning logits into g (16 bits, one piece of it held at
// a time), then one launch with the tiles of both gradient products.
//
// All three products share one kernel: a persistent CTA, or a pair of CTAs on
// one 256 x 256 tile where there are more than 128 rows, walks a list of
// tiles.  A producer warp streams 128-byte wide K blocks of A and B through a
// ring of shared-memory stages (TMA, 128-byte swizzle), one thread issues
// tcgen05.mma into one of two TMEM accumulators, and eight warps work on the
// other one.
//
// What bounds it.  Few rows: reading W, once in the forward pass and twice in
// the backward one (for the logits and for dh), and writing dW.  128 x 768 x
// 131072 bf16: forward 36 us (5.7 TB/s), backward 121 to 131 us from card to
// card (201 MB of W twice, 201 MB of dW, 34 MB of g written and read twice: up
// to 5.8 TB/s).  Many rows: the
// tensor cores.  4096 x 2048 x 128000 bf16: forward 1.1 to 1.2 ms (1.8 to 2.0
// PFLOP/s as the power limit lets the clock), forward and backward 5.13 ms with
// the logits worked out twice (1.67 PFLOP/s).  Between: tiles of a short K,
// whose epilogue takes as long as its product (1024 x 1024 x 50021: forward 65
// us, 1.6 PFLOP/s; backward 208 us).
// Keeping g for a second use in the L2 cache, with both gradients trailing the
// logits inside one launch, was not faster than two launches over pieces of the
// vocabulary (128 x 768 x 131072: 137 to 166 us): a CTA's own turns then add up.
#include <atomic>
#include <cmath>

#include "launch.cuh"
#include "tc_tile.cuh"

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
constexpr int kCeThreads = 32 * (kEpiWarps + 2);
constexpr int kBN = 256;                 // tile columns
constexpr int kJoinThreads = 128;
// K blocks that are summed in the tensor cores' accumulator alone.  It rounds each
// step's sum toward zero, which takes about 6e-9 of a sum of terms of one sign for
// each of them (in one sum, dW of 2^17 rows was 7.6e-4 too small, of 2^20 rows
// 6e-3).  Longer sums are taken in parts, which are added in fp32, rounded to
// nearest.  dW, whose terms may well have one sign, in parts of 16384 rows: 1e-4,
// half of fp16's rounding (40000 x 1024 x 60000 bf16 backward: 11.75 ms, 11.45
// in one sum).  dh, whose terms have the signs of a column of W, in parts of at
// most 65536 labels (with 16384, 777 x 1000 x 50021 backward takes 253 us, not
// 234).
constexpr int kDwBlocks = 256, kDhBlocks = 1024;
constexpr int kMaxSplit = 64;            // parts of dh's K
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
    static constexpr int C = kSMs / CG;            // clusters
};

// kGradLong: kGrad whose dW sums, of more than kDwBlocks K blocks, are taken in parts
enum Mode { kLse = 0, kProb = 1, kGrad = 2, kGradLong = 3 };
constexpr bool is_grad(int mode) { return mode >= kGrad; }

struct CeCtl {
    uint64_t full[6], empty[6], tfull[2], tempty[2];
    uint32_t tmem;
    int abort_flag;
};

struct CeArgs {
    int32_t T, V, H;      // rows, vocabulary, features
    int32_t v0;           // first vocabulary row of the piece
    int32_t nm, nn, nk;   // tiles of the logits (rows, columns of the piece), K blocks
    int32_t bw;           // columns of a tile of logits
    int32_t ab, an;       // rows of a box of A by its rows (h; g in dh's product), and boxes: rows past them
                          // stay unset, and their results unused
    int32_t kt;           // rows of a box of g and h in dW's product, whose K they are
    int32_t f16;          // 16-bit operands are fp16, not bf16
    // kLse
    const float *h_scale, *W_scale;  // fp8: scale per row (W: from row v0 on), or NULL
    const int32_t *targets;
    float2 *part;         // [tile rows][slots] running maximum (of z log2 e) and sum
    float *zsum;          // the same for the sum of z, or NULL
    int32_t slots;
    float *ztgt;          // [T] the target's logit
    int32_t ignore;
    // kProb
    const float *lse, *dloss;
    float *gscale;        // factor of g and its inverse, written by the first CTA
    float smooth, full;   // full: see g_scale
    // kGrad: dh units first (rows x features x pieces of K), then dW tiles
    int32_t nh;           // tiles along H
    int32_t dh_tiles, dh_split, dh_kb, dh_each, dh_hi;  // tiles, pieces of K, K blocks; units of a cluster
    int32_t dw_tiles, dw_hi, dw_lo, dw_nk;
    int32_t dw_segs;      // parts of a dW tile's K
    int32_t first;        // the piece is the first: dh sums start from zero
    float *acc;           // dh sums, [unit][CTA][column / 4][128 rows][4]
    float *dw_acc;        // the same of a cluster's dW tile, where dw_segs > 1
    uint16_t *dW;         // where dW's rows do not suit TMA, else NULL
    int64_t lddW;
    int32_t *status;
};

struct Tile {
    int kind;  // 0: logits, 1: dh, 2: dW
    int m0, n0, k0, nk, unit, seg;
};

// tile i of cluster c
template <int CG, int MODE>
__device__ __forceinline__ bool tile_at(const CeArgs &a, int c, int i, Tile &t)
{
    constexpr int C = Cfg<CG>::C, BM = Cfg<CG>::BM;
    if constexpr (!is_grad(MODE)) {
        // bands of kBand row tiles; inside a band the row tile runs fastest,
        // so W is read from memory once for a band
        const uint32_t l = (uint32_t)i * C + c;
        if (l >= (uint32_t)(a.nm * a.nn))  // below 2^31
            return false;
        const uint32_t per = kBand * a.nn;
        const uint32_t b = a.nm <= kBand ? 0 : l / per, r = l - b * per;
        const uint32_t mc = min(kBand, a.nm - b * kBand);
        const uint32_t n = r / mc;
        t.kind = 0;
        t.m0 = (b * kBand + (r - n * mc)) * BM;
        t.n0 = n * a.bw;
        t.k0 = 0;
        t.nk = a.nk;
        t.unit = n;
        return true;
    } else {
        const uint32_t hi = a.dh_hi;  // clusters below it have one dh unit more
        const uint32_t mine = a.dh_each + ((uint32_t)c < hi ? 1 : 0);
        constexpr bool LONG = MODE == kGradLong;
        if ((uint32_t)i < mine) {
            const uint32_t u = (uint32_t)i * C + c, s = u / (uint32_t)a.dh_tiles, x = u - s * a.dh_tiles;
            const uint32_t m = x / (uint32_t)a.nh;
            t.kind = 1;
            t.m0 = m * BM;
            t.n0 = (x - m * a.nh) * kBN;
            t.k0 = (int)((int64_t)s * a.dh_kb / a.dh_split);
            t.nk = (int)((int64_t)(s + 1) * a.dh_kb / a.dh_split) - t.k0;
            t.unit = u;
            return true;
        }
        const uint32_t jj = (uint32_t)i - mine, segs = LONG ? a.dw_segs : 1, j = LONG ? jj / segs : jj;
        // dW tiles in turn over the clusters; those with one dh unit more take
        // only the first dw_hi turns
        uint32_t l;
        if (j < (uint32_t)a.dw_hi)
            l = j * C + c;
        else if (j < (uint32_t)a.dw_lo && (uint32_t)c >= hi)
            l = a.dw_hi * C + (j - a.dw_hi) * (C - hi) + (c - hi);
        else
            return false;
        if (l >= (uint32_t)a.dw_tiles)
            return false;
        const uint32_t m = l / (uint32_t)a.nh;
        t.kind = 2;
        t.m0 = m * BM;
        t.n0 = (l - m * a.nh) * kBN;
        t.k0 = 0;
        t.nk = a.dw_nk;
        t.unit = 0;
        if (LONG) {
            t.seg = (int)(jj - j * segs);
            t.k0 = (int)((int64_t)a.dw_nk * t.seg / a.dw_segs);
            t.nk = (int)((int64_t)a.dw_nk * (t.seg + 1) / a.dw_segs) - t.k0;
        }
        return true;
    }
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// errors of calls that were given no status word
__device__ int32_t g_ce_status;

__device__ __forceinline__ int32_t *status_of(int32_t *status) { return status ? status : &g_ce_status; }

// whether the row of target y has a loss and a gradient
__device__ __forceinline__ bool is_live(const CeArgs &a, int y) { return y != a.ignore && y >= 0 && y < a.V; }

// Factor of g before it is rounded to 16 bits; the products' epilogues take it
// out again.  It brings the largest |dloss| (1 - e) of the rows that have a
// gradient (what the others hold may be anything), the target's part of g, to
// just `full` (1, or 2^14 in fp16, whose range would not hold dloss = 1 / T
// times a probability).  With the same dloss in every row, as in a mean, all
// targets' parts are then a little below a power of two, where a rounding is
// smallest against its value; without it they would all be rounded the same
// way at wherever 1 / T falls (measured at T = 777, fp16, e = 0.1: 4.3e-4 of
// error in dh instead of 2.7e-4 by the output's own rounding).  The epilogue
// warps of every CTA work it out while the first tile is under way; those of
// the first one report targets that are no labels.
__device__ __forceinline__ float g_scale(const CeArgs &a, float *sm)
{
    float top = 0.f;
    for (int t = threadIdx.x; t < a.T; t += kEpiWarps * 32) {
        const float v = fabsf(a.dloss[t]);
        const int y = a.targets[t];
        if (is_live(a, y)) {
            if (v < INFINITY)
                top = fmaxf(top, v);
        } else if (y != a.ignore && blockIdx.x == 0) {
            sg_flag(status_of(a.status), SG_ERR_DATA);
        }
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

// kLse, kProb: A = m_h, B = m_W, out = m_g (kProb).  kGrad: dh from A = m_g (by
// rows), B = m_W; dW from A = m_gk (by columns), B = m_h, out = m_dW.
template <int CG, int MODE, bool F8>
__global__ void __launch_bounds__(kCeThreads, 1)
    k_ce(const __grid_constant__ CUtensorMap m_h, const __grid_constant__ CUtensorMap m_W,
         const __grid_constant__ CUtensorMap m_g, const __grid_constant__ CUtensorMap m_gk,
         const __grid_constant__ CUtensorMap m_dW, const CeArgs a)
{
    using K = Cfg<CG>;
    constexpr int NS = K::NS;
    constexpr int KE = F8 ? 128 : 64;  // elements of a K block
    constexpr bool LONG = MODE == kGradLong;
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
            for (int i = 0; ok && tile_at<CG, MODE>(a, cl, i, t); ++i) {
                const int am = t.m0 + rank * 128;
                // a pair has more than 128 rows: whole boxes
                const int ab = CG == 2 ? 64 : a.ab, an = CG == 2 ? 2 : a.an, kt = CG == 2 ? 64 : a.kt;
                // the next free stage, which is to receive `bytes` in all CTAs
                auto stage = [&](uint32_t bytes, uint32_t *bar) {
                    ok = mbar_wait(smem_u32(&c.empty[r.i]), r.ph ^ 1u, abort_flag, status_of(a.status));
                    *bar = smem_u32(&c.full[r.i]);
                    if (ok && rank == 0)
                        mbar_arrive_expect_tx(*bar, bytes);
                    if constexpr (CG == 2)
                        *bar = mapa(*bar, 0);
                    return base + (uint32_t)r.i * K::kStage;
                };
                // one loop for each product: the thread has some 500 cycles
                // for a K block
                uint32_t bar;
                if (!is_grad(MODE)) {
                    const int bh = a.bw / 2;  // with two CTAs, B's rows of one; else half of them
                    const int bn = a.v0 + t.n0 + rank * bh;
                    const uint32_t bytes = CG * 128 * (an * ab + a.bw / CG), a2 = ab * 128, b2 = bh * 128;
                    const bool two = an == 2;
                    for (int k = 0; k < t.nk * KE; k += KE, r.next(NS)) {
                        const uint32_t st = stage(bytes, &bar);
                        if (!ok)
                            break;
                        tma_load_2d_cg<CG>(st, &m_h, k, am, bar);
                        if (two)
                            tma_load_2d_cg<CG>(st + a2, &m_h, k, am + ab, bar);
                        tma_load_2d_cg<CG>(st + K::kA, &m_W, k, bn, bar);
                        if (CG == 1)
                            tma_load_2d_cg<CG>(st + K::kA + b2, &m_W, k, bn + bh, bar);
                    }
                } else if (t.kind == 1) {
                    const int bn = t.n0 + rank * 128, k1 = (t.k0 + t.nk) * KE;
                    const uint32_t bytes = CG * 128 * (an * ab + K::BRows), a2 = ab * 128;
                    const bool two = an == 2;
                    for (int k = t.k0 * KE; k < k1; k += KE, r.next(NS)) {
                        const uint32_t st = stage(bytes, &bar);
                        if (!ok)
                            break;
                        tma_load_2d_cg<CG>(st, &m_g, k, am, bar);
                        if (two)
                            tma_load_2d_cg<CG>(st + a2, &m_g, k, am + ab, bar);
#pragma unroll
                        for (int j = 0; j < K::BRows / 64; ++j)
                            tma_load_2d_cg<CG>(st + K::kA + j * kBox, &m_W, bn + 64 * j, a.v0 + k, bar);
                    }
                } else {
                    const int bn = t.n0 + rank * 128;
                    const uint32_t bytes = CG * 128 * (2 + K::BRows / 64) * kt;
                    for (int k = LONG ? t.k0 * KE : 0, k1 = k + t.nk * KE; k < k1; k += KE, r.next(NS)) {
                        const uint32_t st = stage(bytes, &bar);
                        if (!ok)
                            break;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tma_load_2d_cg<CG>(st + j * kBox, &m_gk, am + 64 * j, k, bar);
#pragma unroll
                        for (int j = 0; j < K::BRows / 64; ++j)
                            tma_load_2d_cg<CG>(st + K::kA + j * kBox, &m_h, bn + 64 * j, k, bar);
                    }
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
            for (int i = 0; ok && tile_at<CG, MODE>(a, cl, i, t); ++i) {
                if (t.nk == 0)
                    continue;
                const bool a_mn = t.kind == 2, b_mn = t.kind != 0;
                const int bn = is_grad(MODE) ? kBN : a.bw;
                const uint32_t idesc =
                    F8 || a.f16 ? idesc_f16(K::BM, bn, a_mn, b_mn) : idesc_bf16(K::BM, bn, a_mn, b_mn);
                const OpDesc da(base, a_mn), db(base + K::kA, b_mn);
                const int buf = it & 1;
                ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&c.tempty[buf]),
                                                               ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, status_of(a.status)));
                if (!ok)
                    break;
                tc_fence_after();
                for (int kb = 0; kb < t.nk; ++kb) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_cluster(smem_u32(&c.full[r.i]), r.ph, abort_flag, status_of(a.status)));
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t st = (uint32_t)r.i * (K::kStage / 16);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            if (is_grad(MODE) && CG == 1 && a_mn && ks * 16 >= a.kt)
                                break;
                            mma_cg<CG, F8>(tbase + buf * kBN, da.at(st, ks), db.at(st, ks), idesc,
                                           (kb > 0 || ks > 0) ? 1u : 0u);
                        }
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
    } else {
        // ---------------------------------------------------------- epilogue
        // a warp reads its quarter of the TMEM lanes (tile rows) and one half
        // of the tile's columns; a thread has one row
        const int q = warp & 3, half = warp >> 2;
        const int row_in = rank * 128 + q * 32 + lane;
        uint8_t *stg = dsm + (base - smem_u32(dsm)) + NS * K::kStage + warp * kStgWarp;
        float m2 = -INFINITY, s = 0.f, zs = 0.f;
        [[maybe_unused]] float scale = 1.f;
        if constexpr (MODE == kProb)
            scale = g_scale(a, sm_top);
        if constexpr (is_grad(MODE))
            scale = a.gscale[1];
        int it = 0;
        for (int i = 0; tile_at<CG, MODE>(a, cl, i, t); ++i) {
            if (t.nk == 0)
                continue;
            const int buf = it & 1;
            const int row = t.m0 + row_in;              // row of the tile's A operand
            const int cols = is_grad(MODE) ? kBN / 2 : a.bw / 2;  // of this warp, and the first of them
            const int col0 = t.n0 + half * cols;
            const uint32_t tm = tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kBN + half * cols);
            // what the row needs, before the wait
            int tgt = -1;
            [[maybe_unused]] float cf = 0.f, l2 = 0.f, hs = 1.f;
            if constexpr (!is_grad(MODE)) {
                if (row < a.T) {
                    const int y = a.targets[row];
                    const bool live = is_live(a, y);
                    if (live && y - a.v0 - col0 < cols)
                        tgt = y - a.v0 - col0;  // this warp's column of the target, if it has it
                    if constexpr (MODE == kProb) {
                        l2 = a.lse[row] * kLog2e;
                        if (live)
                            cf = a.dloss[row] * scale;
                        else
                            l2 = INFINITY;
                    } else if constexpr (F8) {
                        hs = a.h_scale ? a.h_scale[row] : 1.f;
                    }
                }
            }
            if (!__all_sync(0xffffffffu,
                            mbar_wait_cluster(smem_u32(&c.tfull[buf]), (uint32_t)(it >> 1) & 1u, abort_flag, status_of(a.status))))
                break;
            tc_fence_after();
            if constexpr (MODE == kLse) {
                const int left = min(cols, a.V - a.v0 - col0);  // columns of this warp that are labels
#pragma unroll 1
                for (int cc = 0; cc < cols; cc += 32) {
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
                    const int64_t at = (int64_t)row * a.slots + t.unit * 2 + half;
                    a.part[at] = make_float2(m2, s);
                    if (a.zsum)
                        a.zsum[at] = zs;
                    m2 = -INFINITY;
                    s = zs = 0.f;
                }
            } else if constexpr (MODE == kProb) {
                const int left = a.V - a.v0 - col0;
                const float off = cf * (a.smooth / (float)a.V), hit = cf * (1.f - a.smooth);
                auto out = [&](float (&v)[32], int cc) {
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
                    // lane 0 has the warp's first row
                    store_box(&m_g, col0 + cc, row, row < a.T, stg + (cc & 32) * (kStgWarp / 64), lane, w);
                };
#pragma unroll 1
                for (int cc = 0; cc < cols; cc += 64) {
                    float v[32], u[32];
                    tmem_ld_chunk2<32>(tm + cc, tm + cc + 32, v, u);
                    out(v, cc);
                    out(u, cc + 32);
                }
            } else {
                // a thread's place among the sums of its unit or tile
                const int mine = (half * (kBN / 8)) * 128 + q * 32 + lane;
                if (t.kind == 1) {
                    float4 *acc = reinterpret_cast<float4 *>(a.acc) +
                                  (int64_t)(t.unit * CG + rank) * (kBN / 4) * 128 + mine;
                    auto out = [&](const float (&v)[32], int cc) {
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            float4 *p = acc + (cc / 4 + x) * 128;
                            float4 o = a.first ? make_float4(0.f, 0.f, 0.f, 0.f) : *p;
                            o.x += v[4 * x];
                            o.y += v[4 * x + 1];
                            o.z += v[4 * x + 2];
                            o.w += v[4 * x + 3];
                            *p = o;
                        }
                    };
#pragma unroll 1
                    for (int cc = 0; cc < kBN / 2; cc += 64) {
                        float v[32], u[32];
                        tmem_ld_chunk2<32>(tm + cc, tm + cc + 32, v, u);
                        out(v, cc);
                        out(u, cc + 32);
                    }
                } else {
                    const int64_t row0 = (int64_t)a.v0 + t.m0 + rank * 128 + q * 32;  // the warp's first row of dW
                    const bool done = !LONG || t.seg == a.dw_segs - 1;
                    auto out = [&](float (&v)[32], int cc) {
                        if constexpr (LONG) {
                            float4 *acc = reinterpret_cast<float4 *>(a.dw_acc) +
                                          (int64_t)(cl * CG + rank) * (kBN / 4) * 128 + mine + (cc / 4) * 128;
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                if (t.seg > 0) {
                                    const float4 o = acc[x * 128];
                                    v[4 * x] += o.x;
                                    v[4 * x + 1] += o.y;
                                    v[4 * x + 2] += o.z;
                                    v[4 * x + 3] += o.w;
                                }
                                if (!done)
                                    acc[x * 128] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                            }
                            if (!done)
                                return;
                        }
                        uint32_t w[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            w[x] = pack16(v[2 * x] * scale, v[2 * x + 1] * scale, a.f16);
                        const int x0 = col0 + cc;
                        if (!a.dW) {
                            store_box(&m_dW, x0, (int)row0, row0 < a.V && x0 < a.H, stg + (cc & 32) * (kStgWarp / 64),
                                      lane, w);
                        } else {
                            // rows on any boundary: through shared memory, so
                            // that a warp writes a row at a time
                            uint32_t *rows = reinterpret_cast<uint32_t *>(stg);
                            __syncwarp();
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                rows[lane * 17 + x] = w[x];
                            __syncwarp();
                            for (int r = 0; r < 32 && row0 + r < a.V; ++r)
                                if (x0 + lane < a.H)
                                    a.dW[(row0 + r) * a.lddW + x0 + lane] =
                                        reinterpret_cast<const uint16_t *>(rows + r * 17)[lane];
                        }
                    };
#pragma unroll 1
                    for (int cc = 0; cc < kBN / 2; cc += 64) {
                        float v[32], u[32];
                        tmem_ld_chunk2<32>(tm + cc, tm + cc + 32, v, u);
                        out(v, cc);
                        out(u, cc + 32);
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
            }
            ++it;
        }
        if constexpr (MODE == kLse) {
            if (a.nm == 1) {
                const int64_t at = (int64_t)row_in * a.slots + cl * 2 + half;
                a.part[at] = make_float2(m2, s);
                if (a.zsum)
                    a.zsum[at] = zs;
            }
        }
        if (lane == 0)
            bulk_wait<0>();
        __syncwarp();
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
    int32_t slots, V, ignore;
    float smooth;
    float2 *run;  // what the pieces of the vocabulary before this one came to
    float *zrun;
    int32_t first, last;  // of the pieces
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
    } else if (y != a.ignore) {
        sg_flag(status_of(a.status), SG_ERR_DATA);
    }
    a.loss[t] = out;
}

// lse and loss of a row, a CTA each, from its partial maxima and sums.  Those
// lie by rows, so that a CTA reads lines (1024 x 1024 x 50021, 392 of them to a
// row: whole forward pass 65 us, 68 with a warp's lanes on neighbouring rows).
__global__ void __launch_bounds__(kJoinThreads) k_ce_join(const JoinArgs a)
{
    constexpr int NW = kJoinThreads / 32;
    __shared__ float sm[3][NW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, t = blockIdx.x;
    const float2 *part = a.part + (int64_t)t * a.slots;
    float m = -INFINITY, s = 0.f, zs = 0.f;
    grid_wait();
    for (int i0 = threadIdx.x; i0 < a.slots; i0 += 4 * kJoinThreads) {
        // four loads under way together
        float2 p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kJoinThreads;
            p[j] = i < a.slots ? part[i] : make_float2(-INFINITY, 0.f);
            if (a.zsum)
                zs += i < a.slots ? a.zsum[(int64_t)t * a.slots + i] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            join_one(m, s, p[j]);
    }
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0)
        sm[0][warp] = top;
    __syncthreads();
    for (int w = 0; w < NW; ++w)
        top = fmaxf(top, sm[0][w]);
    s *= exp2f(m - (top == -INFINITY ? 0.f : top));
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
    if (threadIdx.x == 0) {
        for (int w = 1; w < NW; ++w) {
            s += sm[1][w];
            zs += sm[2][w];
        }
        if (!a.first) {
            join_one(top, s, a.run[t]);
            zs += a.zrun[t];
        }
        if (a.last) {
            join_out(a, t, top, s, zs);
        } else {
            a.run[t] = make_float2(top, s);
            a.zrun[t] = zs;
        }
    }
}

// dh = the sum of its pieces.  A CTA has 32 rows and 32 / PARTS columns; a warp
// four of the columns and every PARTS-th piece, whose loads are under way
// together.  (Many pieces mean few tiles: 23 pieces of 128 x 768 took 14 us
// with one warp to all of a column's pieces.)
template <int CG, int PARTS>
__global__ void __launch_bounds__(256)
    k_ce_dh(const float4 *__restrict__ acc, int tiles, int nn, int split, int T, int H,
            const float *__restrict__ gscale, int f16, uint16_t *__restrict__ dh, int64_t lddh)
{
    constexpr int N4 = 8 / PARTS;  // fours of columns
    __shared__ float4 sm[PARTS][N4][32];
    __shared__ uint32_t rows[32][2 * N4 + 1];  // two columns to a word
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c4 = warp % N4, part = warp / N4;
    const int x = blockIdx.x / (CG * 4), rq = blockIdx.x % (CG * 4);  // tile, 32-row part of it
    const int row0 = x / nn * Cfg<CG>::BM + rq * 32, col0 = x % nn * kBN + blockIdx.y * 4 * N4;
    grid_wait();
    if (row0 >= T || col0 >= H)
        return;
    const float inv = gscale[1];
    const float4 *src =
        acc + (((int64_t)x * CG + rq / 4) * (kBN / 4) + blockIdx.y * N4 + c4) * 128 + (rq & 3) * 32 + lane;
    const int64_t step = (int64_t)tiles * CG * (kBN / 4) * 128;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = part; s < split; s += PARTS) {
        const float4 o = src[s * step];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
    }
    if constexpr (PARTS > 1) {
        sm[part][c4][lane] = v;
        __syncthreads();
        if (part == 0) {
#pragma unroll
            for (int i = 1; i < PARTS; ++i) {
                const float4 o = sm[i][c4][lane];
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
        }
    }
    if (part == 0) {
        rows[lane][c4 * 2] = pack16(v.x * inv, v.y * inv, f16);
        rows[lane][c4 * 2 + 1] = pack16(v.z * inv, v.w * inv, f16);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * 4 * N4; i += 256) {
        const int r = i / (4 * N4), c = i % (4 * N4);
        if (row0 + r < T && col0 + c < H)
            dh[(int64_t)(row0 + r) * lddh + col0 + c] = reinterpret_cast<const uint16_t *>(rows[r])[c];
    }
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
template <int CG, int MODE, bool F8>
sg_status launch_ce(const CUtensorMap &h, const CUtensorMap &W, const CUtensorMap &g, const CUtensorMap &gk,
                    const CUtensorMap &dW, const CeArgs &a, bool after, cudaStream_t st)
{
    // once for each device (one bit of the mask)
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    SG_TRY_CUDA(cudaGetDevice(&dev));
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        SG_TRY_CUDA(cudaFuncSetAttribute(k_ce<CG, MODE, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Cfg<CG>::kSmem));
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch(k_ce<CG, MODE, F8>, dim3(Cfg<CG>::C * CG), kCeThreads, (int)Cfg<CG>::kSmem, CG, after, st, h, W, g,
                  gk, dW, a);
}

// One call's tiles and the places of its work memory
struct Plan {
    int es = 2, CG = 1, BM = 128, C = kSMs;
    bool pack_h = false, pack_W = false;
    int64_t ldp = 0;             // row stride of the packed copies
    int64_t nm = 0, bw = kBN;
    int64_t ab = 64, an = 2, kt = 64;  // boxes: see CeArgs
    // forward: rows of a band, vocabulary of a piece
    int64_t Tb = 0, Vb = 0;
    // backward
    int64_t Vc = 0;              // vocabulary of a piece
    int64_t dh_nn = 0, dh_tiles = 0, split = 1;
    // byte offsets
    int64_t o_h = 0, o_W = 0, o_part = 0, o_zsum = 0, o_ztgt = 0, o_run = 0, o_zrun = 0;
    int64_t o_gs = 0, o_g = 0, o_acc = 0, o_dw = 0, bytes = 0;
};

// Time of a tile or dh unit of nk K blocks, in half K blocks: a tile that is
// shorter than its output takes to reach memory (2 K blocks of a CTA, 4 of a
// pair) costs that, and each has a little of its own.
int64_t tile_cost(int64_t nk, int CG) { return 2 * (nk > 2 * CG ? nk : 2 * CG) + 1; }

// Columns of the forward pass's tiles: the width, a multiple of 16, at which the
// clusters' last turn is fullest.  The time of a tile goes by the rows of W
// that it loads and, with two CTAs, whose tiles are bound by the L2 cache, by
// those of h too; it has a little of its own.  (T = 1, H = 2048, V = 128000:
// 572 tiles of 224 on 152 CTAs take 87 us, 500 of 256 take 90.)
int64_t tile_width(int64_t nm, int64_t V, int CG, int C)
{
    int64_t best = kBN, least = 0;
    for (int64_t w = kBN; w >= 128; w -= 16) {
        const int64_t cost = ceil_div(nm * ceil_div(V, w), C) * (w + (CG == 2 ? 272 : 40));
        if (w == kBN || cost < least) {
            best = w;
            least = cost;
        }
    }
    return best;
}

constexpr int64_t kPartBytes = 256ll << 20;

// partial results of a row in a launch over `rows` rows and `vocab` labels: a
// running one for each half of a cluster's tiles, or, where a cluster meets
// several row tiles, one for each half tile; and of all rows
int64_t slot_count(const Plan &p, int64_t rows, int64_t vocab)
{
    return 2 * (rows <= p.BM ? (int64_t)p.C : ceil_div(vocab, p.bw));
}

int64_t part_count(const Plan &p, int64_t rows, int64_t vocab)
{
    return slot_count(p, rows, vocab) * ceil_div(rows, p.BM) * p.BM;
}

void make_plan(const void *h, int64_t ldh, int64_t T, int64_t H, const void *W, int64_t ldw, int64_t V,
               int32_t dtype, bool backward, Plan *p)
{
    p->es = dtype == SG_E4M3 ? 1 : 2;
    p->CG = T > 128 ? 2 : 1;
    p->BM = 128 * p->CG;
    p->C = kSMs / p->CG;
    p->pack_h = !tma_ok(h, ldh, p->es);
    p->pack_W = !tma_ok(W, ldw, p->es);
    p->ldp = ceil_div(H * p->es, 16) * 16 / p->es;
    p->nm = ceil_div(T, p->BM);
    // only the rows that there are: copying boxes of 64 rows of which few exist
    // takes longer than the rest of a stage (forward pass, T = 1, H = 2048, V =
    // 128000: 103 us with two such boxes, 87 with one of 8)
    if (T <= 128) {
        p->an = T <= 64 ? 1 : 2;
        p->ab = ceil_div(ceil_div(T, p->an), 8) * 8;
    }
    if (T < 64)
        p->kt = ceil_div(T, 16) * 16;
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
        p->bw = tile_width(p->nm, V, p->CG, p->C);
        // The partial results of a band of rows, 12 bytes for a row and half tile,
        // are at most kPartBytes: whole bands of kBand row tiles, which read W once
        // each anyway, and where not one fits, pieces of the vocabulary.
        const int64_t band = kBand * p->BM;
        p->Tb = T;
        p->Vb = V;
        if (part_count(*p, T, V) * 12 > kPartBytes) {
            p->Tb = kPartBytes / 12 / slot_count(*p, T, V) / band * band;
            if (p->Tb == 0) {
                p->Tb = T < band ? T : band;
                p->Vb = kPartBytes / 24 / (ceil_div(p->Tb, p->BM) * p->BM) * p->bw;
                p->o_run = take(p->Tb * 8);
                p->o_zrun = take(p->Tb * 4);
            }
        }
        const int64_t parts = part_count(*p, p->Tb, p->Vb);
        p->o_part = take(parts * 8);
        p->o_zsum = take(parts * 4);
        p->o_ztgt = take(p->Tb * 4);
        return;
    }
    // a piece of g holds at most 256 MB (or 256 labels), whatever V: memory that a training
    // program can spare, and pieces long enough that their ends cost little
    int64_t Vc = (256ll << 20) / 2 / T / kBN * kBN;
    if (Vc < kBN)
        Vc = kBN;
    if (Vc > kMaxSplit * kDhBlocks * 64)
        Vc = kMaxSplit * kDhBlocks * 64;
    if (Vc > ceil_div(V, kBN) * kBN)
        Vc = ceil_div(V, kBN) * kBN;
    p->Vc = Vc;
    p->dh_nn = ceil_div(H, kBN);
    p->dh_tiles = p->nm * p->dh_nn;
    // split K of dh until its units and the dW tiles fill the clusters evenly,
    // and into parts of at most kDhBlocks
    const int64_t kb = ceil_div(V < Vc ? V : Vc, 64), dw = ceil_div(Vc, p->BM) * p->dh_nn * tile_cost(ceil_div(T, 64), p->CG);
    double best = 0;
    const int64_t least = ceil_div(kb, kDhBlocks);
    for (int64_t n = least; n <= kb && n <= kMaxSplit; ++n) {
        const int64_t units = p->dh_tiles * n, cost = tile_cost(ceil_div(kb, n), p->CG) + 2;
        const double even = (double)(units * cost + dw) / p->C;
        const double last = (double)(ceil_div(units, p->C) * cost);
        const double span = (even > last ? even : last) * (1.0 + 0.002 * (double)n);
        if (n == least || span < best) {
            best = span;
            p->split = n;
        }
    }
    p->o_gs = take(8);
    p->o_g = take(T * Vc * 2);
    p->o_acc = take(p->dh_tiles * p->split * p->BM * kBN * 4);
    if (ceil_div(T, 64) > kDwBlocks)
        p->o_dw = take((int64_t)p->C * p->BM * kBN * 4);
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

// whether vectors of 32-bit elements (any of them may be NULL) are aligned to them
template <typename... P>
bool aligned4(const P *...p)
{
    return (((uintptr_t)p | ...) & 3) == 0;
}

template <typename E>
void pack(const void *src, int64_t ld, int64_t rows, int64_t cols, void *dst, int64_t ldd, cudaStream_t st)
{
    const int64_t grid = rows < 152 * 8 ? rows : 152 * 8;
    k_ce_pack<E><<<(unsigned)grid, 256, 0, st>>>(static_cast<const E *>(src), ld, rows, (int)cols,
                                                 static_cast<E *>(dst), ldd);
}

// maps of h and W (mh, mW: in the logits' tiles; mhk, mWk: as K rows), packed
// first where their rows need it; h and ldh become those of the copy then
sg_status operand_maps(const Plan &p, const void *&h, int64_t &ldh, int64_t T, int64_t H, const void *W, int64_t ldw,
                       int64_t V, uint8_t *work, CUtensorMap *mh, CUtensorMap *mW, CUtensorMap *mhk, CUtensorMap *mWk, cudaStream_t st)
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
    if (mhk) {
        CE_TRY(map_of(mhk, h, H, T, ldh, p.es, "h", (uint32_t)p.kt));
        CE_TRY(map_of(mWk, W, H, V, ldw, p.es, "W"));
    }
    CE_TRY(map_of(mh, h, H, T, ldh, p.es, "h", (uint32_t)p.ab));
    return map_of(mW, W, H, V, ldw, p.es, "W", (uint32_t)p.bw / 2);
}

}  // namespace

extern "C" {

sg_status sg_softmax_ce_status(int32_t *code, int32_t clear)
{
    const char *fn = "sg_softmax_ce_status";
    if (!code)
        CE_FAIL(SG_ERR_INVALID, "%s: code is NULL", fn);
    *code = SG_OK;
    SG_TRY_CUDA(cudaDeviceSynchronize());
    SG_TRY_CUDA(cudaMemcpyFromSymbol(code, g_ce_status, sizeof(int32_t)));
    const int32_t none = SG_OK;
    if (clear && *code != SG_OK)
        SG_TRY_CUDA(cudaMemcpyToSymbol(g_ce_status, &none, sizeof(int32_t)));
    return SG_OK;
}

sg_status sg_softmax_ce_work(const void *h, int64_t ldh, int64_t T, int64_t H, const void *W, int64_t ldw, int64_t V,
                             int32_t dtype, int32_t backward, int64_t *bytes)
{
    const char *fn = "sg_softmax_ce_work";
    if (!bytes)
        CE_FAIL(SG_ERR_INVALID, "%s: bytes is NULL", fn);
    CE_TRY(check_ce(fn, h, ldh, T, H, W, ldw, V, dtype, backward != 0));
    Plan p;
    if (T > 0)
        make_plan(h, ldh, T, H, W, ldw, V, dtype, backward != 0, &p);
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
    if (!aligned4(h_scale, W_scale, targets, loss, lse, status))
        CE_FAIL(SG_ERR_INVALID, "%s: a vector or status is not aligned to its elements", fn);
    if ((h_scale || W_scale) && dtype != SG_E4M3)
        CE_FAIL(SG_ERR_INVALID, "%s: scales go with SG_E4M3 rows only", fn);
    if (!(smoothing >= 0.0 && smoothing <= 1.0))
        CE_FAIL(SG_ERR_INVALID, "%s: smoothing=%g is outside [0, 1]", fn, smoothing);
    if (T == 0)
        return SG_OK;
    Plan p;
    make_plan(h, ldh, T, H, W, ldw, V, dtype, false, &p);
    if (!work || work_bytes < p.bytes || ((uintptr_t)work & 255) != 0)
        CE_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_softmax_ce_work), aligned to 256", fn,
                (long long)p.bytes);
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t *w8 = static_cast<uint8_t *>(work);
    CUtensorMap mh, mW;
    CE_TRY(operand_maps(p, h, ldh, T, H, W, ldw, V, w8, &mh, &mW, nullptr, nullptr, st));
    CeArgs a = {};
    a.V = (int32_t)V;
    a.H = (int32_t)H;
    a.bw = (int32_t)p.bw;
    a.ab = (int32_t)p.ab;
    a.an = (int32_t)p.an;
    a.kt = (int32_t)p.kt;
    a.nk = (int32_t)ceil_div(H * p.es, 128);
    a.f16 = dtype == SG_F16;
    a.ignore = ignore_index;
    a.part = reinterpret_cast<float2 *>(w8 + p.o_part);
    a.zsum = smoothing > 0 ? reinterpret_cast<float *>(w8 + p.o_zsum) : nullptr;
    a.ztgt = reinterpret_cast<float *>(w8 + p.o_ztgt);
    a.status = status;
    JoinArgs j = {};
    j.part = a.part, j.zsum = a.zsum, j.ztgt = a.ztgt;
    j.status = status, j.V = a.V, j.ignore = ignore_index;
    j.smooth = (float)smoothing;
    j.run = reinterpret_cast<float2 *>(w8 + p.o_run), j.zrun = reinterpret_cast<float *>(w8 + p.o_zrun);
    for (int64_t t0 = 0; t0 < T; t0 += p.Tb) {
        const int64_t rows = T - t0 < p.Tb ? T - t0 : p.Tb;
        if (p.Tb < T)
            CE_TRY(map_of(&mh, static_cast<const uint8_t *>(h) + t0 * ldh * p.es, H, rows, ldh, p.es, "h",
                          (uint32_t)p.ab));
        a.T = (int32_t)rows;
        a.nm = (int32_t)ceil_div(rows, p.BM);
        a.h_scale = h_scale ? h_scale + t0 : nullptr;
        a.targets = j.targets = targets + t0;
        j.loss = loss + t0, j.lse = lse + t0;
        for (int64_t v0 = 0; v0 < V; v0 += p.Vb) {
            const int64_t vc = V - v0 < p.Vb ? V - v0 : p.Vb;
            const bool after = t0 > 0 || v0 > 0;
            a.v0 = (int32_t)v0;
            a.W_scale = W_scale ? W_scale + v0 : nullptr;
            a.nn = (int32_t)ceil_div(vc, p.bw);
            a.slots = j.slots = (int32_t)slot_count(p, rows, vc);
            j.first = v0 == 0, j.last = v0 + vc == V;
            if (dtype == SG_E4M3)
                CE_TRY(p.CG == 1 ? (launch_ce<1, kLse, true>(mh, mW, mh, mh, mh, a, after, st))
                                 : (launch_ce<2, kLse, true>(mh, mW, mh, mh, mh, a, after, st)));
            else
                CE_TRY(p.CG == 1 ? (launch_ce<1, kLse, false>(mh, mW, mh, mh, mh, a, after, st))
                                 : (launch_ce<2, kLse, false>(mh, mW, mh, mh, mh, a, after, st)));
            CE_TRY(launch(k_ce_join, dim3((unsigned)rows), kJoinThreads, 0, 1, true, st, j));
        }
    }
    return SG_OK;
}

sg_status sg_softmax_ce_bwd(const void *h, int64_t ldh, int64_t T, int64_t H, const void *W, int64_t ldw, int64_t V,
                            int32_t dtype, const int32_t *targets, int32_t ignore_index, double smoothing,
                            const float *lse, const float *dloss, void *dh, int64_t lddh, void *dW, int64_t lddw,
                            void *work, int64_t work_bytes, int32_t *status, void *stream)
{
    const char *fn = "sg_softmax_ce_bwd";
    NvtxRange nvtx_(fn);
    CE_TRY(check_ce(fn, h, ldh, T, H, W, ldw, V, dtype, true));
    if (!W || (T && (!h || !targets || !lse || !dloss || (!dh && !dW))))
        CE_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL", fn);
    if (!aligned4(targets, lse, dloss, status))
        CE_FAIL(SG_ERR_INVALID, "%s: a vector or status is not aligned to its elements", fn);
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
    make_plan(h, ldh, T, H, W, ldw, V, dtype, true, &p);
    if (!work || work_bytes < p.bytes || ((uintptr_t)work & 255) != 0)
        CE_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_softmax_ce_work), aligned to 256", fn,
                (long long)p.bytes);
    uint8_t *w8 = static_cast<uint8_t *>(work);
    CUtensorMap mh, mW, mhk, mWk, mg, mgk, mgs, mdW;
    CE_TRY(operand_maps(p, h, ldh, T, H, W, ldw, V, w8, &mh, &mW, &mhk, &mWk, st));
    // g: [T][Vc], loaded by rows and by columns, stored in boxes of 32 x 32
    CE_TRY(map_of(&mg, w8 + p.o_g, p.Vc, T, p.Vc, 2, "g", (uint32_t)p.ab));
    CE_TRY(map_of(&mgk, w8 + p.o_g, p.Vc, T, p.Vc, 2, "g", (uint32_t)p.kt));
    CE_TRY(map_of(&mgs, w8 + p.o_g, p.Vc, T, p.Vc, 2, "g", 32, true));
    // a TMA store ends on a multiple of 16 bytes: with other widths it would
    // write past a row's end
    const bool dw_tma = dW && tma_ok(dW, lddw, 2) && H % 8 == 0;
    if (dw_tma)
        CE_TRY(map_of(&mdW, dW, H, V, lddw, 2, "dW", 32, true));
    else
        mdW = mgs;
    CeArgs a = {};
    a.T = (int32_t)T;
    a.V = (int32_t)V;
    a.H = (int32_t)H;
    a.nm = (int32_t)p.nm;
    a.bw = (int32_t)p.bw;
    a.ab = (int32_t)p.ab;
    a.an = (int32_t)p.an;
    a.kt = (int32_t)p.kt;
    a.nk = (int32_t)ceil_div(H, 64);
    a.f16 = dtype == SG_F16;
    a.targets = targets;
    a.ignore = ignore_index;
    a.lse = lse;
    a.dloss = dloss;
    a.smooth = (float)smoothing;
    a.nh = (int32_t)p.dh_nn;
    a.dh_split = (int32_t)p.split;
    a.dh_tiles = dh ? (int32_t)p.dh_tiles : 0;
    a.dw_nk = (int32_t)ceil_div(T, 64);
    a.dw_segs = (int32_t)ceil_div(a.dw_nk, kDwBlocks);
    a.acc = reinterpret_cast<float *>(w8 + p.o_acc);
    a.dw_acc = reinterpret_cast<float *>(w8 + p.o_dw);
    a.dW = dW && !dw_tma ? static_cast<uint16_t *>(dW) : nullptr;
    a.lddW = lddw;
    a.status = status;
    a.gscale = reinterpret_cast<float *>(w8 + p.o_gs);
    a.full = dtype == SG_F16 ? 16384.f : 1.f;
    for (int64_t v0 = 0; v0 < V; v0 += p.Vc) {
        const int64_t vc = V - v0 < p.Vc ? V - v0 : p.Vc;
        a.v0 = (int32_t)v0;
        a.first = v0 == 0;
        a.nn = (int32_t)ceil_div(vc, p.bw);
        CE_TRY(p.CG == 1 ? (launch_ce<1, kProb, false>(mh, mW, mgs, mgs, mgs, a, v0 > 0, st))
                         : (launch_ce<2, kProb, false>(mh, mW, mgs, mgs, mgs, a, v0 > 0, st)));
        a.dh_kb = (int32_t)ceil_div(vc, 64);
        a.dw_tiles = dW ? (int32_t)(ceil_div(vc, p.BM) * p.dh_nn) : 0;
        // turns of dW tiles so that all clusters end at about the same time
        const int64_t units = (int64_t)a.dh_tiles * p.split, hi = units % p.C;
        a.dh_each = (int32_t)(units / p.C);
        a.dh_hi = (int32_t)hi;
        const int64_t less = dh ? ceil_div(tile_cost(ceil_div(a.dh_kb, p.split), p.CG) + 2, tile_cost(a.dw_nk, p.CG)) : 0;
        int64_t q_hi = hi ? (a.dw_tiles - less * (p.C - hi)) / p.C : 0;
        if (q_hi < 0)
            q_hi = 0;
        a.dw_hi = (int32_t)q_hi;
        a.dw_lo = (int32_t)(q_hi + ceil_div(a.dw_tiles - q_hi * p.C > 0 ? a.dw_tiles - q_hi * p.C : 0, p.C - hi));
        if (a.dw_segs > 1)  // more than 128 rows: pairs
            CE_TRY((launch_ce<2, kGradLong, false>(mhk, mWk, mg, mgk, mdW, a, true, st)));
        else
            CE_TRY(p.CG == 1 ? (launch_ce<1, kGrad, false>(mhk, mWk, mg, mgk, mdW, a, true, st))
                             : (launch_ce<2, kGrad, false>(mhk, mWk, mg, mgk, mdW, a, true, st)));
    }
    if (dh) {
        const int parts = p.split >= 8 ? 4 : 1;
        const dim3 grid((unsigned)(p.dh_tiles * p.CG * 4), (unsigned)(kBN / 32 * parts));
        const float4 *acc = reinterpret_cast<const float4 *>(a.acc);
        return launch(p.CG == 1 ? (parts == 4 ? k_ce_dh<1, 4> : k_ce_dh<1, 1>)
                                : (parts == 4 ? k_ce_dh<2, 4> : k_ce_dh<2, 1>),
                      grid, 256, 0, 1, true, st, acc, (int)p.dh_tiles, (int)p.dh_nn, (int)p.split, (int)T, (int)H,
                      (const float *)a.gscale, (int)a.f16, static_cast<uint16_t *>(dh), lddh);
    }
    return SG_OK;
}

}  // extern "C"
