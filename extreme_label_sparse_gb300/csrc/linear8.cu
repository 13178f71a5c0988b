// Linear layer on 8-bit integers with a scale for each token and each channel,
// and its gradients (definitions in include/sg.h):
//   out[t][n] = xs[t] ws[n] sum_h x8[t][h] W8[n][h],
//   dx = dout (ws W8),  dW = dout^T (xs x8).
// The integer rate of this chip's tensor cores is far below their 16-bit rate,
// and a product of 16-bit operands loses nothing: an int8 is exact in fp16, a
// product of two is below 2^14, and a sum of 1024 of them at most 2^24, exact in
// an fp32 accumulator.  So the operands are brought to 16 bits first, and after
// 1024 terms an accumulator is added to fp32 sums in registers, rounded to
// nearest (the tensor cores' own sums round toward zero), while the next terms
// go into the other one.
//
// One kernel for the three products: a persistent CTA, or a pair of CTAs on one
// 256 x 256 tile, walks a list of tiles.  A producer warp streams K blocks of 64
// through a ring of shared-memory stages (TMA, 128-byte swizzle), one thread issues
// tcgen05.mma into one of two TMEM accumulators, and eight warps take the sums of
// the other one.  Products of few tiles are split along K, their parts joined in a
// fixed order.  Few tokens go another way (linear8_few.cuh).
//
// What bounds it: the tensor cores.  4096 x 4096 x 16384: 299 us, of which the
// product 262 (2.1 PFLOP/s, 89 % of the tensor pipe's cycles: integers in fp16 draw
// less power than other values, so the clock stays up) and bringing 80 MB of integers
// to 16 bits 37.  Gradients of 8192 x 4096 x 4096: 318 us.
#include <cmath>

#include "linear8_few.cuh"
#include "linear8_turns.cuh"

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kDrain = 16;    // K blocks summed in a TMEM accumulator: 1024 terms

template <int CG>
struct Cfg {
    static constexpr int BM = 128 * CG;  // tile rows
    static constexpr int BRows = kBN / CG;
    static constexpr uint32_t kA = 2 * kBox;  // bytes of A's and B's part of a stage
    static constexpr uint32_t kB = (BRows / 64) * kBox;
    static constexpr uint32_t kStage = kA + kB;
    static constexpr int NS = CG == 2 ? 6 : 4;
    static constexpr uint32_t kSmem = NS * kStage + kEpiWarps * kStgWarp + 1024;
    static constexpr int C = kSMs / CG;  // clusters
};

struct LinCtl {
    uint64_t full[6], empty[6], tfull[2], tempty[2];
    uint32_t tmem;
    int abort_flag;
};

// 16 packed words (32 columns of 16 bits, or 16 of 32) of this warp's 32 rows
// where their rows may start anywhere: through shared memory, so that a warp
// writes pieces of rows
template <int SIZE>
__device__ __forceinline__ void store_rows(const Prod &p, int row0, int x0, uint8_t *stg, int lane,
                                           const uint32_t (&w)[16])
{
    uint32_t *rows = reinterpret_cast<uint32_t *>(stg);
    if (lane == 0)
        bulk_wait_read<0>();  // the other product's outputs may go by store_box
    __syncwarp();
#pragma unroll
    for (int x = 0; x < 16; ++x)
        rows[lane * 17 + x] = w[x];
    __syncwarp();
    // eight pieces under way together
    if constexpr (SIZE == 2) {
        if (x0 + lane < p.N) {
            uint16_t *at = static_cast<uint16_t *>(p.out) + row0 * p.ldo + x0 + lane;
#pragma unroll 8
            for (int r = 0; r < 32; ++r, at += p.ldo)
                if (row0 + r < p.M)
                    *at = (uint16_t)(rows[r * 17 + lane / 2] >> (16 * (lane & 1)));
        }
    } else {
        const int c = lane & 15;
        if (x0 + c < p.N) {
            uint32_t *at = static_cast<uint32_t *>(p.out) + (row0 + lane / 16) * p.ldo + x0 + c;
#pragma unroll 8
            for (int r = lane / 16; r < 32; r += 2, at += 2 * p.ldo)
                if (row0 + r < p.M)
                    *at = rows[r * 17 + c];
        }
    }
}

template <int CG>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear(const __grid_constant__ CUtensorMap mA0, const __grid_constant__ CUtensorMap mB0,
             const __grid_constant__ CUtensorMap mO0, const __grid_constant__ CUtensorMap mA1,
             const __grid_constant__ CUtensorMap mB1, const __grid_constant__ CUtensorMap mO1,
             const __grid_constant__ LinArgs a)
{
    using K = Cfg<CG>;
    constexpr int NS = K::NS;
    __shared__ LinCtl c;
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
    int32_t *status = lin_status(a.status);
    Unit t;

    if (warp == kEpiWarps) {
        // ---------------------------------------------------------- producer
        // the whole warp walks the list, an elected thread copies (see elect_one:
        // by `lane == 0` the copies of a K block took longer than its MMAs)
        Ring r;
        bool ok = true;
        for (int i = 0; ok && unit_at<CG>(a, cl, i, t); ++i) {
            const Prod &p = a.p[t.which];
            const CUtensorMap *mA = t.which ? &mA1 : &mA0, *mB = t.which ? &mB1 : &mB0;
            const int am = t.m0 + rank * 128, bn = t.n0 + rank * 128;
            // a pair has more than 128 rows: whole boxes
            const int ab = CG == 2 ? 128 : a.ab, kt = CG == 2 || !p.a_mn ? 64 : a.kt;
            const uint32_t bytes = CG * 128 * ((p.a_mn ? 2 * kt : ab) + (p.b_mn ? K::BRows / 64 * kt : K::BRows));
            const bool a_mn = p.a_mn, b_mn = p.b_mn;
            for (int k = t.k0 * 64, k1 = k + t.nk * 64; k < k1; k += 64, r.next(NS)) {
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c.empty[r.i]), r.ph ^ 1u, abort_flag, status));
                if (!ok)
                    break;
                if (elect_one()) {
                    uint32_t bar = smem_u32(&c.full[r.i]);
                    if (rank == 0)
                        mbar_arrive_expect_tx(bar, bytes);
                    if constexpr (CG == 2)
                        bar = mapa(bar, 0);
                    const uint32_t st = base + (uint32_t)r.i * K::kStage;
                    if (a_mn) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tma_load_2d_cg<CG>(st + j * kBox, mA, am + 64 * j, k, bar);
                    } else {
                        tma_load_2d_cg<CG>(st, mA, k, am, bar);
                    }
                    if (b_mn) {
#pragma unroll
                        for (int j = 0; j < K::BRows / 64; ++j)
                            tma_load_2d_cg<CG>(st + K::kA + j * kBox, mB, bn + 64 * j, k, bar);
                    } else {
                        tma_load_2d_cg<CG>(st + K::kA, mB, k, bn, bar);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) {
            // gave up: copies may still be on their way into this CTA (and signal
            // the pair's first CTA); they land long before this
            const uint64_t t0 = global_ns();
            while (global_ns() - t0 < 1000000u) {
            }
        }
        __syncwarp();
    } else if (warp == kEpiWarps + 1) {
        // ---------------------------------------------------------- MMA
        if (rank == 0) {
            Ring r;
            int it = 0;
            bool ok = true;
            for (int i = 0; ok && unit_at<CG>(a, cl, i, t); ++i) {
                const Prod &p = a.p[t.which];
                const uint32_t idesc =
                    p.f16 ? idesc_f16(K::BM, kBN, p.a_mn, p.b_mn) : idesc_bf16(K::BM, kBN, p.a_mn, p.b_mn);
                const OpDesc da(base, p.a_mn), db(base + K::kA, p.b_mn);
                const int kt = CG == 2 || !p.a_mn ? 64 : a.kt;
                for (int kb = 0; ok && kb < t.nk; ++it) {
                    const int buf = it & 1, end = min(t.nk, kb + kDrain);
                    ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&c.tempty[buf]),
                                                                   ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, status));
                    if (!ok)
                        break;
                    tc_fence_after();
                    for (int k0 = kb; kb < end; ++kb) {
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait_cluster(smem_u32(&c.full[r.i]), r.ph, abort_flag, status));
                        if (!ok)
                            break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t st = (uint32_t)r.i * (K::kStage / 16);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) {
                                if (CG == 1 && ks * 16 >= kt)
                                    break;
                                mma_cg<CG, false>(tbase + buf * kBN, da.at(st, ks), db.at(st, ks), idesc,
                                                  (kb > k0 || ks > 0) ? 1u : 0u);
                            }
                            mma_commit_cg<CG>(smem_u32(&c.empty[r.i]));
                        }
                        __syncwarp();
                        r.next(NS);
                    }
                    if (ok && elect_one())
                        mma_commit_cg<CG>(smem_u32(&c.tfull[buf]));
                    __syncwarp();
                }
            }
        }
    } else {
        // ---------------------------------------------------------- epilogue
        // a warp reads its quarter of the TMEM lanes (tile rows) and one half
        // of the tile's columns; a thread has one row, whose 128 sums it holds
        const int q = warp & 3, half = warp >> 2;
        uint8_t *stg = dsm + (base - smem_u32(dsm)) + NS * K::kStage + warp * kStgWarp;
        int it = 0, box = 0;
        bool ok = true;
        for (int i = 0; ok && unit_at<CG>(a, cl, i, t); ++i) {
            const Prod &p = a.p[t.which];
            const int row0 = t.m0 + rank * 128 + q * 32, col0 = t.n0 + half * (kBN / 2);  // the warp's first
            float v[4][32];
            for (int kb = 0; kb < t.nk; kb += kDrain, ++it) {
                const int buf = it & 1;
                const uint32_t tm = tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kBN + half * (kBN / 2));
                ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&c.tfull[buf]), (uint32_t)(it >> 1) & 1u,
                                                               abort_flag, status));
                if (!ok)
                    break;
                tc_fence_after();
                if (kb == 0) {
                    tmem_ld_chunk2<32>(tm, tm + 32, v[0], v[1]);
                    tmem_ld_chunk2<32>(tm + 64, tm + 96, v[2], v[3]);
                } else {
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float w[16];
                            tmem_ld_chunk<16>(tm + cc * 32 + h * 16, w);
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                v[cc][16 * h + x] += w[x];
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&c.tempty[buf]);
                    // the accumulator's values are in registers already
                    // (wait::ld): nothing in memory has to be visible with this
                    if constexpr (CG == 2)
                        mbar_arrive_remote_relaxed(mapa(bar, 0));
                    else
                        mbar_arrive(bar);
                }
            }
            if (!ok)
                break;
            if (p.split > 1) {
                float4 *acc = reinterpret_cast<float4 *>(p.acc) + ((int64_t)t.id * CG + rank) * (kBN / 4) * 128 +
                              half * (kBN / 8) * 128 + q * 32 + lane;
#pragma unroll
                for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        acc[(cc * 8 + x) * 128] =
                            make_float4(v[cc][4 * x], v[cc][4 * x + 1], v[cc][4 * x + 2], v[cc][4 * x + 3]);
                continue;
            }
            const CUtensorMap *mO = t.which ? &mO1 : &mO0;
            float rs = p.inv ? *p.inv : 1.f;
            if (p.rs)
                rs = row0 + lane < p.M ? p.rs[row0 + lane] : 0.f;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                const int x0 = col0 + cc * 32;
                if (p.cs) {
                    const float mine = x0 + lane < p.N ? p.cs[x0 + lane] : 0.f;
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        v[cc][x] = v[cc][x] * rs * __shfl_sync(0xffffffffu, mine, x);
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        v[cc][x] *= rs;
                }
                uint32_t w[16];
                if (p.otype == SG_F32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            w[x] = __float_as_uint(v[cc][16 * h + x]);
                        if (p.out)
                            store_rows<4>(p, row0, x0 + 16 * h, stg, lane, w);
                        else
                            store_box(mO, x0 + 16 * h, row0, row0 < p.M && x0 + 16 * h < p.N, stg + (box ^= kStgWarp / 2),
                                      lane, w);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        w[x] = pack16(v[cc][2 * x], v[cc][2 * x + 1], p.otype == SG_F16);
                    if (p.out)
                        store_rows<2>(p, row0, x0, stg, lane, w);
                    else
                        store_box(mO, x0, row0, row0 < p.M && x0 < p.N, stg + (box ^= kStgWarp / 2), lane, w);
                }
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
// The parts of a split product, joined in their order: a CTA has 32 rows and 32
// columns of a tile, a warp four of the columns.
template <int CG>
__global__ void __launch_bounds__(256) k_linear_join(const __grid_constant__ Prod p)
{
    __shared__ float rows[32][33];
    const int lane = threadIdx.x & 31, c4 = threadIdx.x / 32;
    const uint32_t x = blockIdx.x / (CG * 4), rq = blockIdx.x % (CG * 4);  // tile, 32-row part of it
    // the tile's place, as in unit_at
    const uint32_t per = 16u * p.nt, b = x / per, y = x - b * per;
    const uint32_t mc = min(16u, p.mt - b * 16), n = y / mc;
    const int row0 = (int)(b * 16 + (y - n * mc)) * Cfg<CG>::BM + rq * 32, col0 = (int)n * kBN + blockIdx.y * 32;
    grid_wait();
    if (row0 >= p.M || col0 >= p.N)
        return;
    const int64_t step = (int64_t)p.mt * p.nt * CG * (kBN / 4) * 128;
    const float4 *src = reinterpret_cast<const float4 *>(p.acc) +
                        (((int64_t)x * CG + rq / 4) * (kBN / 4) + blockIdx.y * 8 + c4) * 128 + (rq & 3) * 32 + lane;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < p.split; ++s) {
        const float4 o = src[s * step];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
    }
    rows[lane][c4 * 4] = v.x;
    rows[lane][c4 * 4 + 1] = v.y;
    rows[lane][c4 * 4 + 2] = v.z;
    rows[lane][c4 * 4 + 3] = v.w;
    __syncthreads();
    const int col = col0 + lane;
    if (col >= p.N)
        return;
    const float cs = p.cs ? p.cs[col] : p.inv ? *p.inv : 1.f;
    for (int r = c4; r < 32 && row0 + r < p.M; r += 8) {
        const float z = rows[r][lane] * (p.rs ? p.rs[row0 + r] : 1.f) * cs;
        const int64_t at = (row0 + r) * p.ldo + col;
        if (p.otype == SG_F32)
            static_cast<float *>(p.out)[at] = z;
        else if (p.otype == SG_F16)
            static_cast<__half *>(p.out)[at] = __float2half_rn(z);
        else
            static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(z);
    }
}

// factor_of the largest scales of two vectors, by a CTA each
__global__ void __launch_bounds__(1024)
    k_factor(const float *s0, int64_t n0, float *f0, const float *s1, int64_t n1, float *f1)
{
    __shared__ float sm[32];
    const float2 f = factor_of<1024>(blockIdx.x ? s1 : s0, blockIdx.x ? n1 : n0, sm);
    if (threadIdx.x == 0)
        *reinterpret_cast<float2 *>(blockIdx.x ? f1 : f0) = f;
}

// rows that do not start on 16 bytes, copied to a stride that does
__global__ void __launch_bounds__(256)
    k_linear_copy(const uint16_t *__restrict__ src, int64_t ld, int64_t rows, int cols, uint16_t *__restrict__ dst,
                  int64_t ldd)
{
    grid_wait();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += 256)
            dst[r * ldd + c] = src[r * ld + c];
}

// ---------------------------------------------------------------- host
template <int CG>
sg_status launch_linear(const CUtensorMap (&m)[6], const LinArgs &a, cudaStream_t st)
{
    // once for each device (one bit of the mask)
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    SG_TRY_CUDA(cudaGetDevice(&dev));
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        SG_TRY_CUDA(cudaFuncSetAttribute(k_linear<CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<CG>::kSmem));
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    LIN_TRY(launch(k_linear<CG>, dim3(Cfg<CG>::C * CG), kThreads, (int)Cfg<CG>::kSmem, CG, true, st, m[0], m[1], m[2],
                   m[3], m[4], m[5], a));
    for (const Prod &p : a.p)
        if (p.units && p.split > 1)
            LIN_TRY(launch(k_linear_join<CG>, dim3((unsigned)(p.mt * p.nt * CG * 4), kBN / 32), 256, 0, 1, true, st, p));
    return SG_OK;
}

void make_plan(int64_t T, int64_t H, int64_t N, const void *dout, int64_t ldd, bool backward, bool want_dx,
               bool want_dW, Plan *p)
{
    p->ldh = ceil_div(H, 16) * 16;
    p->ldn = ceil_div(N, 8) * 8;
    if (T <= 128)  // boxes of the rows that there are
        p->ab = ceil_div(T, 8) * 8;
    if (T < 64)
        p->kt = ceil_div(T, 16) * 16;
    auto take = [&](int64_t n) {
        const int64_t at = p->bytes;
        p->bytes += ceil_div(n, 256) * 256;
        return at;
    };
    p->o_f = take(16);
    if (!backward) {
        int64_t Nc = kPiece / 2 / p->ldh / kBN * kBN;
        if (Nc < kBN)
            Nc = kBN;
        p->Nc = Nc < N ? Nc : N;
        p->o_x = take(T * p->ldh * 2);
        p->o_W = take(p->Nc * p->ldh * 2);
        choose_tiles(T, H, p->Nc, false, false, false, p);
        // the last piece may be split otherwise: room for either
        int64_t most = 0;
        for (int64_t n : {p->Nc, N % p->Nc}) {
            if (n == 0)
                continue;
            Prod a = {}, none = {};
            shape(a, *p, T, n, H);
            choose_splits(a, none, p->C);
            const int64_t need = a.split > 1 ? (int64_t)a.units * p->BM * kBN * 4 : 0;
            most = need > most ? need : most;
        }
        p->o_acc[0] = take(most);
        return;
    }
    choose_tiles(T, H, N, true, want_dx, want_dW, p);
    p->copy = !tma_ok(dout, ldd, 2);
    p->o_x = take(want_dW ? T * p->ldh * 2 : 0);
    p->o_W = take(want_dx ? N * p->ldh * 2 : 0);
    p->o_d = take(p->copy ? T * p->ldn * 2 : 0);
    for (int i = 0; i < 2; ++i)
        p->o_acc[i] = take(p->p[i].split > 1 ? (int64_t)p->p[i].units * p->BM * kBN * 4 : 0);
}

sg_status check_linear(const char *fn, const int8_t *x8, int64_t ldx, int64_t T, int64_t H, const int8_t *W8, int64_t ldw,
                       int64_t N)
{
    if (T < 0 || H < 1 || N < 1)
        LIN_FAIL(SG_ERR_INVALID, "%s: need T >= 0, H >= 1 and N >= 1 (T=%lld H=%lld N=%lld)", fn, (long long)T,
                 (long long)H, (long long)N);
    // the last: tiles are counted in 31 bits
    if (T > (1 << 24) || H > (1 << 20) || N > (1 << 24) || ceil_div(T, 128) * ceil_div(N, 256) >= (1ll << 28))
        LIN_FAIL(SG_ERR_UNSUPPORTED, "%s: T=%lld, H=%lld, N=%lld or T N is above 2^24, 2^20, 2^24 or 2^43", fn,
                 (long long)T, (long long)H, (long long)N);
    if (ldx < H || ldw < H)
        LIN_FAIL(SG_ERR_INVALID, "%s: a row stride (%lld, %lld) is below H=%lld", fn, (long long)ldx, (long long)ldw,
                 (long long)H);
    return SG_OK;
}

// whether vectors of 32-bit elements (any of them may be NULL) are aligned to them
template <typename... P>
bool aligned4(const P *...p)
{
    return (((uintptr_t)p | ...) & 3) == 0;
}

// map of an output where TMA can write it (a store ends on a multiple of 16
// bytes: with other widths it would go past a row's end)
sg_status out_map(Prod &p, CUtensorMap *m, const CUtensorMap &none, void *out, int64_t ldo, int32_t dtype, const char *name)
{
    const int es = dtype == SG_F32 ? 4 : 2;
    p.otype = dtype;
    p.ldo = ldo;
    p.out = out;
    *m = none;
    if (p.split > 1 || !tma_ok(out, ldo, es) || (int64_t)p.N * es % 16 != 0)
        return SG_OK;
    LIN_TRY(map_of(m, out, p.N, p.M, ldo, es, name, 32, true));
    p.out = nullptr;
    return SG_OK;
}

}  // namespace

extern "C" {

sg_status sg_linear8_status(int32_t *code, int32_t clear)
{
    const char *fn = "sg_linear8_status";
    if (!code)
        LIN_FAIL(SG_ERR_INVALID, "%s: code is NULL", fn);
    *code = SG_OK;
    SG_TRY_CUDA(cudaDeviceSynchronize());
    SG_TRY_CUDA(cudaMemcpyFromSymbol(code, g_linear_status, sizeof(int32_t)));
    const int32_t none = SG_OK;
    if (clear && *code != SG_OK)
        SG_TRY_CUDA(cudaMemcpyToSymbol(g_linear_status, &none, sizeof(int32_t)));
    return SG_OK;
}

sg_status sg_linear8_work(const int8_t *x8, int64_t ldx, int64_t T, int64_t H, const int8_t *W8, int64_t ldw, int64_t N,
                          const void *dout, int64_t lddout, int32_t backward, int64_t *bytes)
{
    const char *fn = "sg_linear8_work";
    if (!bytes)
        LIN_FAIL(SG_ERR_INVALID, "%s: bytes is NULL", fn);
    LIN_TRY(check_linear(fn, x8, ldx, T, H, W8, ldw, N));
    *bytes = 0;
    if (T == 0)
        return SG_OK;
    if (!backward && is_few(T)) {
        *bytes = few_plan(x8, ldx, T, H, W8, ldw, N).bytes;
        return SG_OK;
    }
    // backward: either gradient may be left out, which changes the splits
    for (int i = 0; i < (backward ? 3 : 1); ++i) {
        Plan p;
        make_plan(T, H, N, dout, lddout, backward != 0, i != 1, i != 2, &p);
        *bytes = p.bytes > *bytes ? p.bytes : *bytes;
    }
    return SG_OK;
}

sg_status sg_linear8_fwd(const int8_t *x8, int64_t ldx, const float *x_scale, int64_t T, int64_t H, const int8_t *W8,
                         int64_t ldw, const float *W_scale, int64_t N, void *out, int64_t ldo, int32_t dtype, void *work,
                         int64_t work_bytes, int32_t *status, void *stream)
{
    const char *fn = "sg_linear8_fwd";
    NvtxRange nvtx_(fn);
    LIN_TRY(check_linear(fn, x8, ldx, T, H, W8, ldw, N));
    if (dtype != SG_BF16 && dtype != SG_F16 && dtype != SG_F32)
        LIN_FAIL(SG_ERR_INVALID, "%s: dtype %d is not SG_BF16, SG_F16 or SG_F32", fn, dtype);
    if (!W8 || !W_scale || (T && (!x8 || !x_scale || !out)))
        LIN_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL", fn);
    if (!aligned4(x_scale, W_scale, status))
        LIN_FAIL(SG_ERR_INVALID, "%s: a vector or status is not aligned to its elements", fn);
    const int64_t es = dtype == SG_F32 ? 4 : 2;
    if (ldo < N || (uintptr_t)out % es != 0)
        LIN_FAIL(SG_ERR_INVALID, "%s: out has a row stride below N or is not aligned to its elements", fn);
    if (T == 0)
        return SG_OK;
    Plan pl;
    FewPlan few = {};
    if (is_few(T)) {
        few = few_plan(x8, ldx, T, H, W8, ldw, N);
        pl.bytes = few.bytes;
    } else {
        make_plan(T, H, N, nullptr, 0, false, false, false, &pl);
    }
    if (pl.bytes && (!work || work_bytes < pl.bytes || ((uintptr_t)work & 255) != 0))
        LIN_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_linear8_work), aligned to 256", fn, (long long)pl.bytes);
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t *w8 = static_cast<uint8_t *>(work);
    if (is_few(T))
        return few_fwd(x8, ldx, x_scale, T, H, W8, ldw, W_scale, N, out, ldo, dtype, few, w8, status, st);
    const Widen none = {};
    for (int64_t n0 = 0; n0 < N; n0 += pl.Nc) {
        const int64_t nc = N - n0 < pl.Nc ? N - n0 : pl.Nc;
        LIN_TRY(widen(widen_of(W8 + n0 * ldw, ldw, nc, H, nullptr, 0, nullptr, w8 + pl.o_W, pl.ldh, true),
                      n0 ? none : widen_of(x8, ldx, T, H, nullptr, 0, nullptr, w8 + pl.o_x, pl.ldh, true), n0 > 0, st));
        LinArgs a = {};
        a.ab = (int32_t)pl.ab, a.kt = (int32_t)pl.kt, a.status = status;
        Prod &p = a.p[0];
        shape(p, pl, T, nc, H);
        choose_splits(p, a.p[1], pl.C);
        p.f16 = 1;
        p.rs = x_scale;
        p.cs = W_scale + n0;
        p.acc = reinterpret_cast<float *>(w8 + pl.o_acc[0]);
        CUtensorMap m[6];
        LIN_TRY(map_of(&m[0], w8 + pl.o_x, H, T, pl.ldh, 2, "x", (uint32_t)pl.ab));
        LIN_TRY(map_of(&m[1], w8 + pl.o_W, H, nc, pl.ldh, 2, "W", (uint32_t)(kBN / pl.CG)));
        LIN_TRY(out_map(p, &m[2], m[0], static_cast<uint8_t *>(out) + n0 * es, ldo, dtype, "out"));
        m[3] = m[4] = m[5] = m[0];
        schedule(a, pl.C);
        LIN_TRY(pl.CG == 1 ? launch_linear<1>(m, a, st) : launch_linear<2>(m, a, st));
    }
    return SG_OK;
}

sg_status sg_linear8_bwd(const int8_t *x8, int64_t ldx, const float *x_scale, int32_t x_group, int64_t T, int64_t H,
                         const int8_t *W8, int64_t ldw, const float *W_scale, int64_t N, const void *dout, int64_t lddout,
                         int32_t dtype, void *dx, int64_t lddx, void *dW, int64_t lddw, void *work, int64_t work_bytes,
                         int32_t *status, void *stream)
{
    const char *fn = "sg_linear8_bwd";
    NvtxRange nvtx_(fn);
    LIN_TRY(check_linear(fn, x8, dW ? ldx : H, T, H, W8, dx ? ldw : H, N));
    if (dtype != SG_BF16 && dtype != SG_F16)
        LIN_FAIL(SG_ERR_INVALID, "%s: dtype %d is not SG_BF16 or SG_F16", fn, dtype);
    if (x_group != 0 && x_group != rows::kGroup)
        LIN_FAIL(SG_ERR_INVALID, "%s: x_group=%d is not 0 (the row) or %d", fn, x_group, rows::kGroup);
    if (T && (!dout || (!dx && !dW) || (dx && (!W8 || !W_scale)) || (dW && (!x8 || !x_scale))))
        LIN_FAIL(SG_ERR_INVALID, "%s: a required pointer is NULL", fn);
    if (!aligned4(x_scale, W_scale, status))
        LIN_FAIL(SG_ERR_INVALID, "%s: a vector or status is not aligned to its elements", fn);
    if (T && (lddout < N || (uintptr_t)dout % 2 != 0))
        LIN_FAIL(SG_ERR_INVALID, "%s: dout has a row stride below N or is not aligned to its elements", fn);
    if ((dx && (lddx < H || (uintptr_t)dx % 2 != 0)) || (dW && (lddw < H || (uintptr_t)dW % 2 != 0)))
        LIN_FAIL(SG_ERR_INVALID, "%s: dx or dW has a row stride below H or is not aligned to its elements", fn);
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {
        if (dW)
            SG_TRY_CUDA(cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)H * 2, (size_t)N, st));
        return SG_OK;
    }
    Plan pl;
    make_plan(T, H, N, dout, lddout, true, dx != nullptr, dW != nullptr, &pl);
    if (!work || work_bytes < pl.bytes || ((uintptr_t)work & 255) != 0)
        LIN_FAIL(SG_ERR_INVALID, "%s: work needs %lld bytes (sg_linear8_work), aligned to 256", fn, (long long)pl.bytes);
    uint8_t *w8 = static_cast<uint8_t *>(work);
    const bool f16 = dtype == SG_F16;
    // factors of the scales: fp16 has not their range
    float *fac = f16 ? reinterpret_cast<float *>(w8 + pl.o_f) : nullptr;
    const int64_t nW = dx ? N : 0, nx = dW ? T * (x_group ? ceil_div(H, (int64_t)x_group) : 1) : 0;
    // by the kernel that widens, where each of its threads has at most 24 scales to
    // look at: a launch less (whole calls of 128 x 768 x 3000, 5003 and 5800: 26, 29
    // and 27 us for 32, 33 and 32).  Each CTA reads them all, so that the kernels alone
    // win up to 3000 (18.2 us for 19.0), lose 1.4 us at 5800, and 6 at 11000: in a
    // captured graph, where a launch costs the CPU nothing, above 4000 that is lost.
    const bool with = f16 && nW + nx <= 24 * 256;
    bool after = false;  // this call's kernels have begun
    if (f16 && !with) {
        k_factor<<<2, 1024, 0, st>>>(W_scale, nW, fac, x_scale, nx, fac + 2);
        SG_TRY_CUDA(cudaGetLastError());
        after = true;
    }
    if (pl.copy) {
        LIN_TRY(launch(k_linear_copy, dim3((unsigned)(T < kSMs * 8 ? T : kSMs * 8)), 256, 0, 1, after, st,
                       static_cast<const uint16_t *>(dout), lddout, T, (int)N,
                       reinterpret_cast<uint16_t *>(w8 + pl.o_d), pl.ldn));
        dout = w8 + pl.o_d;
        lddout = pl.ldn;
        after = true;
    }
    Widen wide[2] = {};
    if (dx)
        wide[0] = widen_of(W8, ldw, N, H, W_scale, 0, fac, w8 + pl.o_W, pl.ldh, f16, with ? nW : 0);
    if (dW)
        wide[1] = widen_of(x8, ldx, T, H, x_scale, x_group, fac ? fac + 2 : nullptr, w8 + pl.o_x, pl.ldh, f16,
                           with ? nx : 0);
    LIN_TRY(widen(wide[0], wide[1], after, st));
    LinArgs a = {};
    a.p[0] = pl.p[0], a.p[1] = pl.p[1];
    a.ab = (int32_t)pl.ab, a.kt = (int32_t)pl.kt, a.status = status;
    CUtensorMap m[6];
    for (int i = 0; i < 2; ++i) {
        Prod &p = a.p[i];
        CUtensorMap *mi = m + 3 * i;
        const bool is_dW = p.a_mn;
        if (!p.units) {
            mi[0] = mi[1] = mi[2] = m[0];
            continue;
        }
        p.f16 = f16;
        p.acc = reinterpret_cast<float *>(w8 + pl.o_acc[i]);
        p.b_mn = 1;
        p.inv = fac ? fac + (is_dW ? 3 : 1) : nullptr;
        LIN_TRY(map_of(&mi[0], dout, N, T, lddout, 2, "dout", (uint32_t)(is_dW ? pl.kt : pl.ab)));
        if (is_dW)
            LIN_TRY(map_of(&mi[1], w8 + pl.o_x, H, T, pl.ldh, 2, "x", (uint32_t)pl.kt));
        else
            LIN_TRY(map_of(&mi[1], w8 + pl.o_W, H, N, pl.ldh, 2, "W"));
        LIN_TRY(out_map(p, &mi[2], mi[0], is_dW ? dW : dx, is_dW ? lddw : lddx, dtype, is_dW ? "dW" : "dx"));
    }
    schedule(a, pl.C);
    return pl.CG == 1 ? launch_linear<1>(m, a, st) : launch_linear<2>(m, a, st);
}

}  // extern "C"
