// The tiles of the 8-bit linear layer's products: their sizes, how they are cut along
// K, and which cluster has which.  Plain C++, so that the dealing out can be walked
// through without a GPU.
#pragma once

#include <cstdint>
#include <utility>

#ifdef __CUDACC__
#include "linear8_widen.cuh"
#define LIN_BOTH __host__ __device__ __forceinline__
#else  // by itself
#define LIN_BOTH inline
constexpr int kSMs = 152;
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
#endif

namespace {

constexpr int kBN = 256;      // tile columns

// out = A B^T: operands stored with K along their rows, or (mn) with K rows
struct Prod {
    int32_t a_mn, b_mn;
    int32_t M, N;            // of the output
    int32_t mt, nt, nk;      // tiles, K blocks
    int32_t split, units;    // parts of K; tiles times parts
    int32_t f16;             // operands are fp16, not bf16
    int32_t otype;           // sg_dtype of the output
    void *out;               // where its rows do not suit TMA, else NULL
    int64_t ldo;
    const float *rs, *cs;    // factors of its rows and columns, or NULL
    const float *inv;        // factor of all, or NULL
    float *acc;              // parts, [unit][CTA][column / 4][128 rows][4], where split > 1
};

struct LinArgs {
    Prod p[2];
    // units of the first product in turn over the clusters, `each` to each and
    // one more to the first `hi`, which take only b_hi turns of the second's
    int32_t each, hi, b_hi, b_lo;
    int32_t ab;      // rows of a box of A by its rows
    int32_t kt;      // rows of a box whose rows are K, where those are the tokens
    int32_t *status;
};

struct Unit {
    int which, m0, n0, k0, nk, id;
};

// unit i of cluster c
template <int CG>
LIN_BOTH bool unit_at(const LinArgs &a, int c, int i, Unit &t)
{
    constexpr int C = kSMs / CG, BM = 128 * CG;
    const int mine = a.each + (c < a.hi ? 1 : 0);
    uint32_t u;
    t.which = i >= mine;
    if (i < mine) {
        u = (uint32_t)i * C + c;
    } else {
        const int j = i - mine;
        if (j < a.b_hi)
            u = (uint32_t)j * C + c;
        else if (j < a.b_lo && c >= a.hi)
            u = (uint32_t)a.b_hi * C + (uint32_t)(j - a.b_hi) * (C - a.hi) + (c - a.hi);
        else
            return false;
    }
    const Prod &p = a.p[t.which];
    if (u >= (uint32_t)p.units)
        return false;
    // the parts of K run slowest, the row tiles fastest inside bands of 16 of
    // them: what the clusters read at one time stays in the L2 cache
    const uint32_t tiles = (uint32_t)p.mt * p.nt, s = u / tiles;
    uint32_t x = u - s * tiles;
    const uint32_t per = 16u * p.nt, b = x / per;
    x -= b * per;
    const uint32_t left = p.mt - b * 16, mc = left < 16 ? left : 16, n = x / mc;
    t.m0 = (int)(b * 16 + (x - n * mc)) * BM;
    t.n0 = (int)n * kBN;
    t.k0 = (int)((int64_t)s * p.nk / p.split);
    t.nk = (int)((int64_t)(s + 1) * p.nk / p.split) - t.k0;
    t.id = (int)u;
    return true;
}

// Time of a unit of nk K blocks, in K blocks: its own, and an end that the
// other units' work hides in part; a part of a split tile is written, read and
// joined in fp32.
double unit_cost(int64_t nk, bool split) { return (double)nk + (split ? 10.0 : 2.0); }

constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 40, 48, 64};

// parts of K of the products (the second may have no tiles) so that the
// clusters end early; the time that they take, in K blocks
double choose_splits(Prod &a, Prod &b, int C)
{
    const int64_t ta = (int64_t)a.mt * a.nt, tb = (int64_t)b.mt * b.nt;
    double best = -1;
    int sa = 1, sb = 1;
    for (int i : kSplits) {
        if (i > 1 && (i > a.nk || ta * i > 4 * C))
            break;
        for (int j : kSplits) {
            if (j > 1 && (j > b.nk || tb * j > 4 * C || !tb))
                break;
            const double ca = unit_cost(ceil_div(a.nk, i), i > 1), cb = unit_cost(ceil_div(b.nk, j), j > 1);
            const double na = (double)(ta * i), nb = (double)(tb * j);
            const double even = (na * ca + nb * cb) / C;
            // what the longest cluster has of each alone
            const double la = (double)ceil_div(ta * i, C) * ca, lb = (double)ceil_div(tb * j, C) * cb;
            double span = even > la ? even : la;
            if (lb > span)
                span = lb;
            span += 0.5 * ((even > la && even > lb) ? (ca > cb ? ca : cb) * 0.3 : 0.0) + (i > 1 ? 2.0 + 0.1 * i : 0) +
                    (j > 1 ? 2.0 + 0.1 * j : 0);
            if (best < 0 || span < best) {
                best = span;
                sa = i;
                sb = j;
            }
        }
    }
    a.split = sa;
    b.split = sb;
    a.units = (int32_t)(ta * sa);
    b.units = (int32_t)(tb * sb);
    return best;
}

// Time of a unit in its cluster, in K blocks: the next unit's products hide the
// end of one that is as long as its own output takes to be written, of 16 bits
// or of a part's 32.
double unit_time(const Prod &p)
{
    const double nk = (double)ceil_div(p.nk, p.split), out = p.split > 1 ? 8.0 : 4.0;
    return (nk > out ? nk : out) + 2.0;
}

// Turns of the second product's units: b_hi in every cluster, b_lo in those that
// have one of the first's less, so that the last cluster ends first of all the
// choices; that end, in K blocks.  (Rounding the balance of the two down instead
// gave 12 pairs three long units each at 2048 x 1024 x 4096 and the other 64 none:
// 64 us for 30.)
double turns(const Prod &a, const Prod &b, int C, int32_t *b_hi, int32_t *b_lo)
{
    const int64_t na = a.units, nb = b.units, each = na / C, hi = na % C;
    const double ca = na ? unit_time(a) : 0, cb = nb ? unit_time(b) : 0;
    double best = -1;
    for (int64_t q = hi ? 0 : nb / C, top = hi ? ceil_div(nb, (int64_t)C) : q; q <= top; ++q) {
        const int64_t rest = nb - q * C, lo = q + (rest > 0 ? ceil_div(rest, C - hi) : 0);
        const double t_hi = hi ? (double)(each + 1) * ca + (double)q * cb : 0;
        const double t_lo = (double)each * ca + (double)lo * cb, end = t_hi > t_lo ? t_hi : t_lo;
        if (best < 0 || end < best) {
            best = end;
            *b_hi = (int32_t)q;
            *b_lo = (int32_t)lo;
        }
        // more in every cluster only ends later from here on
        if (t_hi >= t_lo)
            break;
    }
    return best;
}

void schedule(LinArgs &a, int C)
{
    a.each = a.p[0].units / C;
    a.hi = a.p[0].units % C;
    turns(a.p[0], a.p[1], C, &a.b_hi, &a.b_lo);
}

// One call's tiles and the places of its work memory
struct Plan {
    int CG = 1, BM = 128, C = kSMs;
    int64_t ldh = 0, ldn = 0;  // row strides of the copies
    int64_t ab = 128, kt = 64;
    int64_t Nc = 0;            // forward: channels of a piece
    bool copy = false;         // of dout
    Prod p[2] = {};
    int64_t o_f = 0, o_x = 0, o_W = 0, o_d = 0, o_acc[2] = {0, 0}, bytes = 0;
};

void shape(Prod &p, const Plan &pl, int64_t M, int64_t N, int64_t Kd)
{
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.mt = (int32_t)ceil_div(M, pl.BM);
    p.nt = (int32_t)ceil_div(N, kBN);
    p.nk = (int32_t)ceil_div(Kd, 64);
}

// CTAs or pairs of them, and the products' tiles and splits: pairs read less from
// the L2 cache for a tile, CTAs alone have finer turns (777 x 1001 x 5003: 140
// tiles in one turn, where 80 of pairs take two).  N: channels, of a piece where
// the forward pass takes several.
void choose_tiles(int64_t T, int64_t H, int64_t N, bool backward, bool want_dx, bool want_dW, Plan *p)
{
    double best = 0;
    for (int cg = 1; cg <= (T > 128 ? 2 : 1); ++cg) {
        Plan q = *p;
        q.CG = cg;
        q.BM = 128 * cg;
        q.C = kSMs / cg;
        q.p[0] = q.p[1] = Prod{};
        if (!backward) {
            shape(q.p[0], q, T, N, H);
        } else {
            if (want_dW) {
                shape(q.p[0], q, N, H, T);
                q.p[0].a_mn = 1;
            }
            if (want_dx)
                shape(q.p[want_dW ? 1 : 0], q, T, H, N);
        }
        const double span = choose_splits(q.p[0], q.p[1], q.C) * (cg == 1 ? 1.1 : 1.0);
        if (cg == 1 || span < best) {
            best = span;
            *p = q;
        }
    }
    // dx first where that ends a tenth earlier (512 x 4096 x 4096 bf16: 36 us for
    // 44); dW first where they end about together: its writes then go beside dx's
    // long loads (64 x 4096 x 4096: 30 us for 34)
    if (p->p[0].units && p->p[1].units) {
        int32_t hi, lo;
        if (turns(p->p[1], p->p[0], p->C, &hi, &lo) < 0.9 * turns(p->p[0], p->p[1], p->C, &hi, &lo))
            std::swap(p->p[0], p->p[1]);
    }
}

}  // namespace
