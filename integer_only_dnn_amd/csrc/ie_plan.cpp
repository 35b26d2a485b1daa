// Host-side planning of the (C, e) library (see ie_plan.h): argument checks,
// convolution geometry, product plans and workspace layouts.  No GPU code.
#include "ie_plan.h"

#include <stdio.h>
#include <stdlib.h>
#include <string.h>

namespace ie {

// ---------------------------------------------------------------------------
// Argument checks and geometry
// ---------------------------------------------------------------------------

int n_exps(const ie_mat *t) { return t->group == IE_GROUP_ROW ? (int)t->rows : 1; }

ie_status check_mat(const ie_mat *t) {
    if (!t) return IE_ERR_NULL;
    if (t->group != IE_GROUP_TENSOR && t->group != IE_GROUP_ROW) return IE_ERR_GROUP;
    if (t->rows < 0 || t->cols < 0 || t->rows > DIM_MAX || t->cols > DIM_MAX) return IE_ERR_SHAPE;
    if (t->rows * t->cols > 0 && !t->mant) return IE_ERR_NULL;
    if ((t->group == IE_GROUP_TENSOR || t->rows > 0) && !t->exp) return IE_ERR_NULL;
    if (t->bits != 0 && (t->bits < 2 || t->bits > 8)) return IE_ERR_BITS;
    return IE_OK;
}

int mat_q(const ie_mat *t) { return (t->bits ? t->bits : 8) - 1; }

FastDiv make_fastdiv(uint32_t d) {
    int l = 0;
    while ((1ull << l) < d) ++l;  // l = ceil(log2 d)
    int s = 31 + l;
    uint64_t m = ((1ull << s) + d - 1) / d;
    return FastDiv{(uint32_t)m, s};
}

ie_status check_conv(const ie_conv_desc *d) {
    if (!d) return IE_ERR_NULL;
    if (d->n < 0 || d->h <= 0 || d->w <= 0 || d->c <= 0 || d->k <= 0 || d->r <= 0 || d->s <= 0 ||
        d->stride <= 0 || d->pad < 0)
        return IE_ERR_SHAPE;
    if ((long long)d->h + 2ll * d->pad < d->r || (long long)d->w + 2ll * d->pad < d->s) return IE_ERR_SHAPE;
    long long rsc = (long long)d->r * d->s * d->c;
    if (rsc > DIM_MAX || (long long)d->n * d->h * d->w * d->c > DIM_MAX * 8ll) return IE_ERR_SHAPE;
    return IE_OK;
}

// Every field is computed in checked 64-bit arithmetic; g.ok is cleared when
// an intermediate overflows or a field does not fit the 32-bit integers the
// kernels use (conv_fits then rejects the shape).
namespace {
struct Checked {
    bool ok = true;
    long long mul(long long a, long long b) {
        long long r = 0;
        if (__builtin_mul_overflow(a, b, &r)) ok = false;
        return ok ? r : 0;
    }
    long long add(long long a, long long b) {
        long long r = 0;
        if (__builtin_add_overflow(a, b, &r)) ok = false;
        return ok ? r : 0;
    }
    long long sub(long long a, long long b) {
        long long r = 0;
        if (__builtin_sub_overflow(a, b, &r)) ok = false;
        return ok ? r : 0;
    }
    int fit(long long v) {
        if (v < -(1ll << 31) || v > DIM_MAX) ok = false;
        return ok ? (int)v : 0;
    }
};
}  // namespace

ConvGeom geom(const ie_conv_desc *d) {
    ConvGeom g;
    memset(&g, 0, sizeof g);
    Checked k;
    auto fdv = [&](long long v) -> FastDiv { return make_fastdiv(v >= 1 && v <= DIM_MAX ? (uint32_t)v : 1u); };
    const long long n = d->n, h = d->h, w = d->w, c = d->c, ko = d->k, r = d->r, s = d->s, st = d->stride,
                    pad = d->pad;
    g.n = d->n;
    g.h = d->h;
    g.w = d->w;
    g.c = d->c;
    g.k = d->k;
    g.r = d->r;
    g.s = d->s;
    g.stride = d->stride;
    g.pad = d->pad;
    // check_conv guarantees h + 2 pad >= r, w + 2 pad >= s and positive sizes
    const long long p = k.sub(k.add(h, k.mul(2, pad)), r) / st + 1;
    const long long q = k.sub(k.add(w, k.mul(2, pad)), s) / st + 1;
    const long long cp = r16(c), kp = r16(ko);
    const long long pq = k.mul(p, q), hw = k.mul(h, w);
    g.p = k.fit(p);
    g.q = k.fit(q);
    g.cp = k.fit(cp);
    g.kp = k.fit(kp);
    k.fit(pq);
    k.fit(hw);
    k.fit(k.mul(n, pq));
    if (!k.ok) return g;  // g.ok stays 0
    g.dpq = fdv(pq);
    g.dq = fdv(q);
    g.dhw = fdv(hw);
    g.dw = fdv(w);
    g.dc = fdv(cp);
    g.ds = fdv(s);
    g.dk = fdv(kp);
    g.dst = fdv(st);
    long long t = BK / cp;
    g.im_dc = k.fit(BK % cp);
    g.im_ds = k.fit(t % s);
    g.im_dr = k.fit(t / s);
    g.im_d0 = k.fit(k.add(k.add(BK % cp, k.mul(t % s, cp)), k.mul(k.mul(t / s, w), cp)));
    g.im_d1 = k.fit(k.mul(w - s, cp));
    t = BK / kp;
    g.dg_dc = k.fit(BK % kp);
    g.dg_ds = k.fit(t % s);
    g.dg_dr = k.fit(t / s);
    const long long rsc = k.mul(k.mul(r, s), c);
    g.wt_d0 = k.fit(k.add(k.mul(BK % kp, rsc), k.mul(t, c)));
    g.wt_d1 = k.fit(k.sub(c, k.mul(kp, rsc)));
    const long long img = k.mul(hw, cp);
    const long long px_dq = BK % q, px_dp = (BK / q) % p;
    g.px_dq = k.fit(px_dq);
    g.px_dp = k.fit(px_dp);
    g.px_d0 = k.fit(k.add(k.add(k.mul(k.mul(px_dq, st), cp), k.mul(k.mul(k.mul(px_dp, st), w), cp)),
                          k.mul(BK / pq, img)));
    g.px_d1 = k.fit(k.mul(k.sub(k.mul(st, w), k.mul(q, st)), cp));
    g.px_d2 = k.fit(k.sub(img, k.mul(k.mul(k.mul(p, st), w), cp)));
    g.px_nw = k.fit(BK / pq + 2);
    g.st_inv = k.fit((65536 + st - 1) / st);
    k.fit(img);
    k.fit(k.mul(pq, kp));
    k.fit(k.mul(k.mul(r, s), cp));
    k.fit(k.mul(k.mul(r, s), kp));
    g.ok = k.ok ? 1 : 0;
    return g;
}

bool conv_fits(const ConvGeom &g) {
    if (!g.ok) return false;
    if (g.r > 15 || g.s > 15 || g.h > 65535 || g.w > 65535 || g.cp > (1 << 22) || g.kp > (1 << 22)) return false;
    const long long pq = (long long)g.p * g.q, hw = (long long)g.h * g.w;
    const long long img_x = hw * g.cp, img_y = pq * g.kp;
    if ((256 / pq + 2) * img_x > WINDOW) return false;  // forward im2col rows, weight-gradient pixels
    if ((256 / hw + 2) * img_y > WINDOW) return false;  // input-gradient gather
    const long long rs = (long long)g.r * g.s;
    return 256 * rs * g.cp <= WINDOW && 256 * rs * g.kp <= WINDOW && 128ll * g.kp <= WINDOW;
}

bool weight_window_fits(const ConvGeom &g) { return (long long)g.kp * g.r * g.s * g.c <= WINDOW; }

// ---------------------------------------------------------------------------
// Stride phases of the input gradient
// ---------------------------------------------------------------------------

bool phases_apply(const ConvGeom &g) {
    if (!conv_fits(g) || g.stride != 2 || g.n <= 0) return false;
    // a phase's tile of at most 256 rows spans at most 256 / (hn wn) + 2
    // output images (as the whole convolution's does)
    const long long img_y = (long long)g.p * g.q * g.kp;
    for (int ph = 0; ph < 2; ++ph)
        for (int pw = 0; pw < 2; ++pw) {
            const long long hn = (g.h - ph + 1) / 2, wn = (g.w - pw + 1) / 2;
            if (hn * wn > 0 && (256 / (hn * wn) + 2) * img_y > WINDOW) return false;
        }
    return true;
}

Phases make_phases(const ConvGeom &g, int bm) {
    Phases ps;
    memset(&ps, 0, sizeof ps);
    if (!phases_apply(g) || bm <= 0) return ps;
    const int st = g.stride;
    ps.n = st * st;
    ps.st = st;
    ps.h = g.h;
    ps.w = g.w;
    int tap = 0, tiles = 0;  // tiles: the most tile rows of one phase
    for (int t = 0; t < ps.n; ++t) {
        PhaseRec &p = ps.r[t];
        p.ph = t / st;
        p.pw = t % st;
        p.hn = g.h > p.ph ? (g.h - p.ph + st - 1) / st : 0;
        p.wn = g.w > p.pw ? (g.w - p.pw + st - 1) / st : 0;
        const int r0 = (p.ph + g.pad) % st, s0 = (p.pw + g.pad) % st;
        p.ra = g.r > r0 ? (g.r - r0 + st - 1) / st : 0;
        p.sb = g.s > s0 ? (g.s - s0 + st - 1) / st : 0;
        p.ch = (p.ph + g.pad - r0) / st;
        p.cw = (p.pw + g.pad - s0) / st;
        const int sb = p.sb > 0 ? p.sb : 1;
        p.ds = (BK / g.kp) % sb;
        p.dr = (BK / g.kp) / sb;
        p.tap0 = tap;
        p.k0 = tap * g.kp;
        p.klen = p.ra * p.sb * g.kp;
        tap += p.ra * p.sb;
        p.rows = g.n * p.hn * p.wn;
        if (cdiv(p.rows, bm) > tiles) tiles = cdiv(p.rows, bm);
        p.dhw = make_fastdiv(p.hn * p.wn > 0 ? (uint32_t)(p.hn * p.wn) : 1u);
        p.dw = make_fastdiv(p.wn > 0 ? (uint32_t)p.wn : 1u);
        p.dsb = make_fastdiv((uint32_t)sb);
        if (p.klen > ps.kmax) ps.kmax = p.klen;
    }
    ps.tm = ps.n * tiles;
    return ps;
}

int phase_tap(const Phases &ps, const ConvGeom &g, int r, int s) {
    const int st = ps.st;
    const int ph = ((r - g.pad) % st + st) % st, pw = ((s - g.pad) % st + st) % st;
    const PhaseRec &p = ps.r[ph * st + pw];
    return p.tap0 + (r / st) * p.sb + s / st;
}

// ---------------------------------------------------------------------------
// Built tiles
// ---------------------------------------------------------------------------

bool tile_built(int family, Tile t, bool partial) {
#define IE_HAS(a, b) \
    if (t.mi == a && t.ni == b) return true;
    switch (family) {
        case FAM_DENSE:
            IE_TILES_DENSE(IE_HAS)
            return false;
        case FAM_ADD:
            if (partial) return tile_built(FAM_DENSE, t, true);
            IE_TILES_ADD(IE_HAS)
            return false;
        case FAM_IM2COL:
        case FAM_DGRAD:
        case FAM_DGRAD_WT:
            IE_TILES_CONV(IE_HAS)
            return false;
        case FAM_WGRAD:
        case FAM_WGRAD_CONV:
            if (!partial) return false;
            IE_TILES_WGRAD(IE_HAS)
            return false;
    }
#undef IE_HAS
    return false;
}

bool pair_tiles_built(Tile t1, Tile t2) {
#define IE_HAS(a, b, c, d) \
    if (t1.mi == a && t1.ni == b && t2.mi == c && t2.ni == d) return true;
    IE_TILES_PAIR(IE_HAS)
#undef IE_HAS
    return false;
}

// ---------------------------------------------------------------------------
// Plans
// ---------------------------------------------------------------------------

// Planning rules, calibrated by timing every plan of the ResNet-18 and ViT-B
// products on an MI355X:
//  * a workgroup runs MI*NI waves' worth of 32x32 MFMA tiles and keeps its
//    loads in flight for a few steps, so small grids are latency bound: the
//    128x128 tile pays off only with at least four workgroups per CU (and a
//    full tile width), 128x64 with two, otherwise 64x64;
//  * a split contraction costs an extra pass over splits x M x N int32
//    partials, so products split only when even 64x64 tiles leave most CUs
//    idle;
//  * weight gradients (short outputs, long contractions) split into chunks
//    of at least eight steps, doubling while fewer than 2.25 workgroups per
//    CU result.
constexpr long long WG_TARGET = 576;

int chunk_for(long long K, int splits) {
    long long c = (K + splits - 1) / splits;
    c = (c + BK - 1) / BK * BK;
    return (int)(c > 0 ? c : BK);
}

Force force_from_env(const char *var, bool wgrad) {
    Force f{0, 0, 0, -1, 1};
    const char *v = getenv(var);
    if (!v || !*v) return f;
    int mi = 0, ni = 0, a = -1, b = 1;
    if (wgrad) {
        if (sscanf(v, "%d,%d,%d", &mi, &ni, &b) != 3) return f;
        a = PLAN_SPLIT;
    } else if (sscanf(v, "%d,%d,%d,%d", &mi, &ni, &a, &b) < 2) {
        return f;
    }
    f.on = 1;
    f.mi = mi;
    f.ni = ni;
    f.mode = a < 0 ? PLAN_RTO : a;
    f.splits = b;
    return f;
}

static Plan forced(const Force &f, long long K) {
    Plan p;
    p.t = Tile{f.mi, f.ni};
    p.mode = f.mode;
    const int sp = f.splits < 1 ? 1 : (f.splits > 4096 ? 4096 : f.splits);
    p.k_chunk = chunk_for(K, sp);
    p.splits = (int)((K + p.k_chunk - 1) / p.k_chunk);
    if (p.splits < 1) p.splits = 1;
    return p;
}

Plan plan_product(long long M, long long N, long long K, int row_group, int family, const Force &f) {
    if (f.on) return forced(f, K);
    auto tiles = [&](Tile t) { return (long long)cdiv(M, t.bm()) * cdiv(N, t.bn()); };
    // Rows of 129..256 results: the 64 x 256 tile holds a whole row group,
    // so its epilogue rounds straight to int8 in one pass.  Measured against
    // the plans below over row-grouped products (bit-identical results): it
    // wins while its tiles need at most two workgroups per CU (M up to
    // 32768; 25216 x 192 x 192: 18.9 vs 25.5 us, x 768: 25.7 vs 29.5 us;
    // 8192 x 192 x 768: 14.6 vs 20.2 us), and loses with more rows (one
    // workgroup per CU: 50432 x 192 x 576, 46.2 vs 40.6 us).  A few tiles
    // with a long contraction keep the split plan below.
    const bool few_long = tiles(Tile{1, 1}) < NCU / 2 && K >= 8 * BK;
    if (row_group && N > 128 && N <= 256 && !few_long && tile_built(family, Tile{1, 4}, false) &&
        tiles(Tile{1, 4}) <= 2ll * NCU)
        return Plan{Tile{1, 4}, PLAN_DIRECT, 1, chunk_for(K, 1)};
    // The 128 x 128 tile for outputs wider than 64 with at least 3/4 of a
    // tile per CU (its matrix work per LDS byte and per barrier is twice the
    // 128 x 64 tile's), else 128 x 64 with 1.5 tiles per CU, else 64 x 64: a
    // sweep of every built tile over the ResNet-50 and ResNet-18 forward and
    // input-gradient products (the smallest ResNet-18 layers, 2048 rows,
    // want the 64 x 64 tile's 512 workgroups).
    Tile t{1, 1};
    if (N > 64 && tiles(Tile{2, 2}) >= 3ll * NCU / 4) t = Tile{2, 2};
    else if (tiles(Tile{2, 1}) >= 3ll * NCU / 2) t = Tile{2, 1};
    const bool direct = row_group ? N <= t.bn() : tiles(t) == 1;
    // Recompute (two passes over the operands) or round to odd (one pass, an
    // int16 round trip of the output): row groups recompute contractions up
    // to RECOMP_KMAX; a whole-tensor result recomputes one-step contractions,
    // and two-step ones whose output is at least twice as wide as the
    // contraction (measured over ResNet-50's forward and input-gradient
    // products: elsewhere the second pass's matrix work outweighs the int16
    // round trip).
    const bool recomp = row_group ? K <= RECOMP_KMAX : K <= BK || (K <= 2 * BK && N >= 2 * K);
    Plan best{t, direct ? PLAN_DIRECT : recomp ? PLAN_RECOMP : PLAN_RTO, 1, chunk_for(K, 1)};
    if (!direct && few_long) {
        const long long n11 = tiles(Tile{1, 1});
        int sp = 1;
        while (sp < 16 && n11 * sp * 2 <= WG_TARGET && K / (sp * 2) >= 4 * BK) sp *= 2;
        if (sp > 1) {
            const int kc = chunk_for(K, sp);
            best = Plan{Tile{1, 1}, PLAN_SPLIT, (int)((K + kc - 1) / kc), kc};
        }
    }
    return best;
}

// One 128 x 128 tile over a short contraction rounds in its own pass: over 64 x
// 128 x 256, 65 x 66 x 16, 65 x 65 x 256, 128 x 64 x 256 and 128 x 128 x 16, 64
// and 256, both groupings, 6.8 to 7.4 us a call; in 64 x 64 tiles with the pass
// that closes them 9.7 to 10.4.  100 x 100 x 200, whose rows are padded first,
// 10.3 and 12.7.
static bool one_tile(long long M, long long N, long long K) { return M <= 128 && N <= 128 && K <= 256; }

Plan plan_add(long long M, long long N, long long K, int row_group, const Force &f) {
    if (!f.on && one_tile(M, N, K) && (M > 64 || N > 64)) return Plan{Tile{2, 2}, PLAN_DIRECT, 1, chunk_for(K, 1)};
    Plan p = plan_product(M, N, K, row_group, FAM_ADD, f);
    if (!f.on && p.mode == PLAN_RECOMP) p.mode = PLAN_RTO;
    return p;
}

// Rows of 129..1024 results and contractions up to 2048 (a narrower row fits
// the tiles' direct form: 100000 x 64 x 256, 11.9 us there, 20.4 here; over a
// longer contraction the weight, streamed again for every 64 rows, takes what
// the second pass cost: 25216 x 768 x 4096, 111 us here, 116 there, 8192 x 1024
// x 4096, 71 and 53), from as many rows on as take the tiles longer than one
// workgroup: x 768 x 192, 10.4 us here at 2048 rows, 12.7 by tiles; x 768 x 768,
// 20.2 here at 6144 rows, 25.0 by tiles, but 20.0 and 19.3 at 4096.
int rows_plan(long long M, long long N, long long K, int row_group, const Force &f) {
    if (f.on || !row_group || N <= 128 || N > 1024 || K < 16 || K > 2048) return 0;
    return M >= (K <= 256 || N <= 256 ? 2048 : 6144) ? cdiv(N, 256) : 0;
}

// Up to 64 rows, unless their results are so many that the tiles fill the chip
// (64 x 32000 x 768: 35.8 us here, 29.3 by tiles; 64 x 4096 x 4096: 16.3 and
// 28.4; 5 x 4096 x 4096: 9.7 and 23.8) or so few columns are so long that
// splitting them fills more of it (8 x 128 x 16384: 16.6 here, 12.3 split; 4 x
// 512 x 8192: 10.6 and 12.4), except at up to 16 rows of a single tile, which is
// not split (8 x 64 x 8192: 11.0 here, 18.6 there; 64 x 64 x 8192: 23.1 and
// 18.7); one tile's worth is left to one launch.
bool few_plan(long long M, long long N, long long K, const Force &f) {
    return !f.on && M <= FEW_ROWS && K >= 16 && M * N <= 1 << 18 && (K <= 32 * N || (M <= 16 && N <= 64)) &&
           !one_tile(M, N, K);
}

DgradPlan plan_dgrad(const ConvGeom &g, int row_group, const Force &f, bool weight_in_place) {
    DgradPlan d;
    memset(&d, 0, sizeof d);
    d.M = (long long)g.n * g.h * g.w;
    d.K = (long long)g.r * g.s * g.kp;
    d.pl = plan_product(d.M, g.c, d.K, row_group, FAM_DGRAD, f);
    const bool want = f.on ? f.mode == PLAN_RECOMP : d.pl.mode != PLAN_DIRECT && !weight_in_place;
    if (row_group || !want || d.M == 0 || !phases_apply(g)) return d;
    d.ps = make_phases(g, d.pl.t.bm());
    if (d.ps.n == 0) return d;
    d.M = (long long)d.ps.tm * d.pl.t.bm();
    d.K = d.ps.kmax;
    d.pl = Plan{d.pl.t, PLAN_RECOMP, 1, chunk_for(d.K, 1)};
    return d;
}

Plan plan_wgrad(long long M, long long N, long long L, int family, const Force &f) {
    (void)family;
    if (f.on) {
        Plan p = forced(f, L);
        p.mode = PLAN_SPLIT;
        return p;
    }
    // The 128 x 128 tile whenever both sides fill it (16 matrix instructions
    // per wave and step, against 4 for the contraction-sliced 64 x 64 one),
    // and about one workgroup per CU in all (two per CU for more than four
    // 64 x 64 tiles): measured over ResNet-50's weight gradients, longer
    // contraction chunks beat a fuller grid, as the split partials (written,
    // then summed by the finalize) shrink with the split count.
    const bool big = M >= 128 && N >= 128;
    const Tile t = big ? Tile{2, 2} : Tile{1, 1};
    const long long nt = (long long)cdiv(M, t.bm()) * cdiv(N, t.bn());
    const long long target = big || nt <= 4 ? NCU : 2 * NCU;
    const int smin = (int)((L + SPLIT_MAX_ROWS - 1) / SPLIT_MAX_ROWS);
    long long want = (target + nt / 2) / nt;  // nearest split count to the target
    const long long smax = L / (8 * BK);      // chunks of at least eight steps
    if (want > smax) want = smax;
    if (want > 1024) want = 1024;
    int sp = want > 1 ? (int)want : 1;
    if (sp < smin) sp = smin;
    const int kc = chunk_for(L, sp);
    const int n = (int)((L + kc - 1) / kc);
    return Plan{t, PLAN_SPLIT, n > 0 ? n : 1, kc};
}

// Tiles built for the batched kernel: 128x128, 64x256, 128x64, 64x64 (the
// 64x256 one for A . B^T only).  A row group fits one tile (direct epilogue,
// no second pass) when N <= the tile width, so rows up to 256 wide take the
// 64x256 tile when there is work enough for it.
Plan plan_batched(long long Z, long long M, long long N, bool kk) {
    auto tiles = [&](Tile t) { return Z * cdiv(M, t.bm()) * cdiv(N, t.bn()); };
    Tile t{1, 1};
    if (kk && N > 128 && N <= 256 && tiles(Tile{1, 4}) >= 2ll * NCU) t = Tile{1, 4};
    else if (N > 64 && tiles(Tile{2, 2}) >= 2ll * NCU) t = Tile{2, 2};
    else if (tiles(Tile{2, 1}) >= 2ll * NCU) t = Tile{2, 1};
    return Plan{t, N <= t.bn() ? PLAN_DIRECT : PLAN_RTO, 1, BK};
}

int recomp_grid(long long M, long long N, long long K, Tile t) {
    const long long tiles = (long long)cdiv(M, t.bm()) * cdiv(N, t.bn());
    // workgroups per CU of the tile's kernel (its one-step form for K <= BK)
    const long long per_cu = K <= BK ? (t.mi * t.ni <= 2 ? 4 : t.mi * t.ni == 4 ? 3 : t.mi * t.ni <= 8 ? 2 : 1)
                                     : (t.mi * t.ni == 1 ? 3 : t.mi * t.ni <= 4 ? 2 : 1);
    long long g = NCU * per_cu;
    if (tiles < g) g = tiles;
    return (int)(g > 8 ? g / 8 * 8 : g);  // a multiple of 8: item % 8 stays the XCD
}

bool plan_valid(const Plan &pl, long long M, long long N, long long K, int row_group, int family) {
    if (pl.t.mi < 1 || pl.t.ni < 1) return false;
    if (pl.mode != PLAN_DIRECT && pl.mode != PLAN_RTO && pl.mode != PLAN_SPLIT && pl.mode != PLAN_RECOMP)
        return false;
    const bool wg = family == FAM_WGRAD || family == FAM_WGRAD_CONV;
    if (wg && pl.mode != PLAN_SPLIT) return false;
    if (family == FAM_ADD && pl.mode == PLAN_RECOMP) return false;
    if (!tile_built(family, pl.t, pl.mode == PLAN_SPLIT)) return false;
    if (pl.splits < 1 || pl.k_chunk <= 0 || pl.k_chunk % BK != 0) return false;
    if ((long long)pl.splits * pl.k_chunk < K) return false;
    if (pl.mode != PLAN_SPLIT && pl.splits != 1) return false;
    if (pl.mode == PLAN_SPLIT && pl.k_chunk > SPLIT_MAX_ROWS) return false;
    const long long tiles = (long long)cdiv(M, pl.t.bm()) * cdiv(N, pl.t.bn());
    if (tiles * pl.splits >= (1ll << 31)) return false;
    if (pl.mode == PLAN_DIRECT && (row_group ? N > pl.t.bn() : tiles > 1)) return false;
    return true;
}

bool plan_valid_batched(const Plan &pl, int form, long long M, long long N, long long K) {
    (void)M;
    const Tile t = pl.t;
    bool built = false;
    if (form == BMM_NT) {
        built = (t.mi == 2 && t.ni == 2) || (t.mi == 1 && t.ni == 4) || (t.mi == 2 && t.ni == 1) ||
                (t.mi == 1 && t.ni == 1);
    } else {
        built = (t.mi == 2 && t.ni == 2) || (t.mi == 2 && t.ni == 1) || (t.mi == 1 && t.ni == 1);
    }
    if (!built || pl.splits != 1 || pl.k_chunk != BK || K > MAX_CONTRACT) return false;
    if (pl.mode == PLAN_DIRECT) return N <= t.bn();
    return pl.mode == PLAN_RTO;
}

// ---------------------------------------------------------------------------
// Workspace
// ---------------------------------------------------------------------------

// One split finalize block per row: 512 threads with up to 4 chunks each.
bool split_round_rows_fits(int Nout, int mc, int mcp) {
    const int vw = (mc == mcp && Nout % 4 == 0) ? 4 : 1;
    return Nout / vw <= SR_THR * SR_MAXV;
}

static size_t mx(size_t a, size_t b) { return a > b ? a : b; }

Needs product_needs(const Plan &pl, long long M, long long N, long long K, int row_group) {
    Needs n{0, 0, 0, 0, 0, 0};
    if (pl.t.mi < 1 || pl.t.ni < 1) return n;
    if (pl.mode == PLAN_RECOMP) {
        n.tneed = row_group ? (size_t)M * cdiv(N, pl.t.bn()) : (size_t)recomp_grid(M, N, K, pl.t);
    } else if (pl.mode == PLAN_RTO) {
        n.p16 = row_group ? (size_t)M * cdiv(N, pl.t.bn()) : (size_t)cdiv(M, pl.t.bm()) * cdiv(N, pl.t.bn());
        n.v16 = (size_t)M * N;
    } else if (pl.mode == PLAN_SPLIT) {
        n.partial = (size_t)pl.splits * M * N;
        if (!(row_group && split_round_rows_fits((int)N, 1, 1))) {
            n.sums = (size_t)M * N;
            n.gneed = row_group ? (size_t)M : 1;
        }
    }
    return n;
}

// The split finalize with bias and residual keeps no sums.
Needs add_needs(const Plan &pl, long long M, long long N, long long K, int row_group) {
    Needs n = product_needs(pl, M, N, K, row_group);
    n.gneed = n.sums = n.tneed = 0;
    if (n.v16) n.v16 = (size_t)M * add_pitch((int)N);
    return n;
}

Needs wgrad_needs(const Plan &pl, long long N, long long Kg, long long Kout, int mc, int mcp, int row_group) {
    Needs n{0, 0, 0, 0, 0, 0};
    n.partial = (size_t)(pl.splits < 1 ? 1 : pl.splits) * N * Kg;
    n.gneed = row_group ? (size_t)N : 1;
    if (!(row_group && split_round_rows_fits((int)Kout, mc, mcp))) n.sums = (size_t)N * Kg;
    return n;
}

Needs batched_needs(const Plan &pl, long long Z, long long M, long long N) {
    Needs n{0, 0, 0, 0, 0, 0};
    if (pl.mode == PLAN_RTO && pl.t.ni >= 1) {
        n.p16 = (size_t)Z * M * cdiv(N, pl.t.bn());
        n.v16 = (size_t)Z * M * N;
    }
    return n;
}

bool covers(const Needs &have, const Needs &need) {
    return need.gneed <= have.gneed && need.p16 <= have.p16 && need.v16 <= have.v16 &&
           need.partial <= have.partial && need.sums <= have.sums && need.tneed <= have.tneed;
}

ProductWs carve_product(Carve &c, long long M, long long N, long long K, int family, const Force &f,
                        size_t tneed_min) {
    ProductWs w{};
    Needs n{0, 0, 0, 0, 0, tneed_min};
    for (int rg = 0; rg < 2; ++rg) {
        const Needs r = product_needs(plan_product(M, N, K, rg, family, f), M, N, K, rg);
        n.gneed = mx(n.gneed, r.gneed);
        n.p16 = mx(n.p16, r.p16);
        n.v16 = mx(n.v16, r.v16);
        n.partial = mx(n.partial, r.partial);
        n.sums = mx(n.sums, r.sums);
        n.tneed = mx(n.tneed, r.tneed);
    }
    n.gneed = mx(n.gneed, M > 0 ? (size_t)M : 1);
    w.gneed = c.take<int>(n.gneed);
    w.p16 = c.take<int16_t>(n.p16);
    w.v16 = c.take<int16_t>(n.v16);
    w.partial = c.take<int>(n.partial);
    w.sums = c.take<long long>(n.sums);
    w.tneed = c.take<int>(n.tneed);
    w.n = n;
    return w;
}

WgradWs carve_wgrad(Carve &c, long long N, long long Kg, long long L, int family, const Force &f) {
    WgradWs w{};
    const Plan pl = plan_wgrad(N, Kg, L, family, f);
    Needs n{0, 0, 0, 0, 0, 0};
    n.gneed = N > 0 ? (size_t)N : 1;
    n.partial = (size_t)(pl.splits < 1 ? 1 : pl.splits) * N * Kg;
    n.sums = (size_t)N * Kg;
    w.eps = c.take<int>(2);
    w.gneed = c.take<int>(n.gneed);
    w.partial = c.take<int>(n.partial);
    w.sums = c.take<long long>(n.sums);
    w.n = n;
    return w;
}

LinearFwdWs carve_linear_fwd(Carve &c, long long M, long long N, long long K, const Force &f) {
    LinearFwdWs w{};
    const long long Kp = r16(K);
    if (Kp != K) {
        w.xp = c.take<int8_t>((size_t)M * Kp);
        w.wp = c.take<int8_t>((size_t)N * Kp);
    }
    w.pw = carve_product(c, M, N, Kp, FAM_DENSE, f);
    return w;
}

LinearFusedWs carve_linear_fused(Carve &c, long long M, long long N, long long K, const Force &f) {
    LinearFusedWs w{};
    const long long Kp = r16(K);
    if (Kp != K) {
        w.l.xp = c.take<int8_t>((size_t)M * Kp);
        w.l.wp = c.take<int8_t>((size_t)N * Kp);
    }
    Needs n{0, 0, 0, 0, 0, 0};
    for (int rg = 0; rg < 2; ++rg) {
        const Needs r = add_needs(plan_add(M, N, Kp, rg, f), M, N, Kp, rg);
        n.p16 = mx(n.p16, r.p16);
        n.v16 = mx(n.v16, r.v16);
        n.partial = mx(n.partial, r.partial);
    }
    w.l.pw.p16 = c.take<int16_t>(n.p16);
    w.l.pw.v16 = c.take<int16_t>(n.v16);
    w.l.pw.partial = c.take<int>(n.partial);
    w.l.pw.n = n;
    w.bmax = c.take<int>(SPLIT_ADD_BLOCKS);
    if (few_plan(M, N, Kp, f)) {
        w.few_acc = c.take<int>((size_t)M * r16(N));
        w.few_w = c.take<int>((size_t)M * (r16(N) / 16));
    }
    if (const int ni = rows_plan(M, N, Kp, 1, f)) w.wt = c.take<int8_t>(rows_weight(ni, Kp));
    return w;
}

LinearDxWs carve_linear_dx(Carve &c, long long M, long long N, long long K, const Force &f) {
    LinearDxWs w{};
    const long long Np = r16(N);
    w.estar = c.take<int>(1);
    w.wt = c.take<int8_t>((size_t)K * Np);
    if (Np != N) w.dyp = c.take<int8_t>((size_t)M * Np);
    w.pw = carve_product(c, M, K, Np, FAM_DENSE, f);
    return w;
}

LinearDwWs carve_linear_dw(Carve &c, long long M, long long N, long long K, const Force &fw) {
    LinearDwWs w{};
    w.dya = c.take<int8_t>((size_t)M * r16(N));
    w.xa = c.take<int8_t>((size_t)M * r16(K));
    w.w = carve_wgrad(c, N, K, M, FAM_WGRAD, fw);
    return w;
}

ConvFwdWs carve_conv_fwd(Carve &c, const ConvGeom &g, const Force &f) {
    ConvFwdWs w{};
    if (g.cp != g.c) {
        w.xp = c.take<int8_t>((size_t)g.n * g.h * g.w * g.cp);
        w.wp = c.take<int8_t>((size_t)g.k * g.r * g.s * g.cp);
    }
    w.pw = carve_product(c, (long long)g.n * g.p * g.q, g.k, (long long)g.r * g.s * g.cp, FAM_IM2COL, f);
    return w;
}

ConvBwdWs carve_conv_bwd(Carve &c, const ConvGeom &g, const Force &f, const Force &fw) {
    ConvBwdWs w{};
    const long long nhw = (long long)g.n * g.h * g.w, npq = (long long)g.n * g.p * g.q;
    w.estar = c.take<int>(1);
    w.wt = c.take<int8_t>((size_t)g.c * g.r * g.s * g.kp);
    if (g.kp != g.k) w.dyp = c.take<int8_t>((size_t)npq * g.kp);
    if (g.cp != g.c) w.xp = c.take<int8_t>((size_t)nhw * g.cp);
    const DgradPlan dp = plan_dgrad(g, 0, f);
    const size_t tn = dp.ps.n ? product_needs(dp.pl, dp.M, g.c, dp.K, 0).tneed : 0;
    w.pw = carve_product(c, nhw, g.c, (long long)g.r * g.s * g.kp, FAM_DGRAD, f, tn);
    w.w = carve_wgrad(c, g.k, (long long)g.r * g.s * g.cp, npq, FAM_WGRAD_CONV, fw);
    return w;
}

BmmWs carve_bmm(Carve &c, int form, long long Z, long long M, long long N, long long K) {
    BmmWs w{};
    const long long Kp = r16(K);
    if (form == BMM_NT) {
        if (Kp != K) {
            w.a = c.take<int8_t>((size_t)(Z * M * Kp));
            w.b = c.take<int8_t>((size_t)(Z * N * Kp));
        }
    } else if (form == BMM_NN) {
        if (Kp != K) w.a = c.take<int8_t>((size_t)(Z * M * Kp));
        w.b = c.take<int8_t>((size_t)(Z * K * r16(N)));
        w.eb = c.take<int>((size_t)(Z > 0 ? Z : 1));
    } else {
        w.a = c.take<int8_t>((size_t)(Z * K * r16(M)));
        w.b = c.take<int8_t>((size_t)(Z * K * r16(N)));
        w.ea = c.take<int>((size_t)(Z > 0 ? Z : 1));
        w.eb = c.take<int>((size_t)(Z > 0 ? Z : 1));
    }
    // round-to-odd values and per-(row, column tile) needs, when the plan
    // rounds in two passes
    w.n = batched_needs(plan_batched(Z, M, N, form == BMM_NT), Z, M, N);
    if (w.n.p16) {
        w.p16 = c.take<int16_t>(w.n.p16);
        w.v16 = c.take<int16_t>(w.n.v16);
    }
    return w;
}

bool is_vector(const ie_mat *t, long long n) {
    return (t->rows == n && t->cols == 1) || (t->rows == 1 && t->cols == n);
}

namespace {
struct RowShape {
    int t, e;
};
// The first of the shapes (in ascending order of t * e) that holds a row.
RowShape first_fit(const RowShape *s, int n, long long cols) {
    for (int i = 0; i + 1 < n; ++i)
        if (cols <= (long long)s[i].t * s[i].e) return s[i];
    return s[n - 1];
}
}  // namespace

// Rows of up to 768 elements take 16 threads (four rows share a wave, its
// reductions and its square root), longer ones a wave or a block.  With few
// rows (NORM_FEW) more threads per row make the shorter chain of work (3000 x
// 768: 4.9 us with 32 threads, 5.4 with 16; 25216 x 768: 15.1 and 14.7), but at
// 1025 to 2048 columns the 256 threads that few rows take are no gain (500 x
// 1500: 5.4 us, 5.3 with 64) or a loss (2000 x 1100: 9.7 and 6.0; 4000 x 2040:
// 16.2 and 9.9).  As
// many blocks as are resident, two or four a CU by their registers, so that
// each keeps its parameters for several rows (25216 x 768 at 512, 1024 and 2048
// blocks: 14.7, 15.2, 16.8 us; 50432 x 192: 11.5, 10.9, 12.5).
NormPlan norm_fwd_plan(long long rows, long long cols) {
    static const RowShape many[] = {{16, 4},  {16, 8},  {16, 12}, {16, 16},  {16, 24},  {16, 32},   {16, 48}, {64, 16},
                                    {64, 24}, {64, 32}, {64, 48}, {256, 16}, {256, 24}, {1024, 8}, {1024, 12}, {1024, 16}};
    static const RowShape few[] = {{64, 4},   {64, 8},   {32, 24},  {64, 16}, {256, 12},
                                   {256, 16}, {256, 24}, {1024, 8}, {1024, 12}, {1024, 16}};
    const RowShape s = rows >= NORM_FEW ? first_fit(many, sizeof many / sizeof *many, cols)
                                        : first_fit(few, sizeof few / sizeof *few, cols);
    const long long rpb = s.t > 256 ? 1 : 256 / s.t, want = (rows + rpb - 1) / rpb;
    const long long cap = s.t >= 256 || s.e > 24 ? 2 * NCU : 4 * NCU;
    return NormPlan{s.t, s.e, (int)(want < 1 ? 1 : want > cap ? cap : want)};
}

NormPlan norm_one_plan(long long rows, long long cols) {
    static const RowShape tall[] = {{16, 4}, {16, 8}, {16, 12}, {16, 16}}, flat[] = {{64, 4}, {64, 8}, {64, 16}};
    if (rows <= 16 && cols <= 1024) {
        const RowShape s = first_fit(flat, 3, cols);
        return NormPlan{s.t, s.e, 1};
    }
    if (rows <= 64 && cols <= 256) {
        const RowShape s = first_fit(tall, 4, cols);
        return NormPlan{s.t, s.e, 1};
    }
    return NormPlan{0, 0, 0};
}

// Each thread keeps the column sums of its elements, so at most 16; blocks of
// 512 threads (of one row when it takes more than 64), eight waves a CU, each
// block leaving one row of partial sums (50432 x 192 in 128, 256 and 512
// blocks: 37.2, 26.4, 30.7 us; 4096 x 4096 in 256 and 512 of 256 threads: 56.3
// and 46.5, but 898 x 2327, mostly its partial sums, 20.2 and 23.2).
NormPlan norm_bwd_plan(long long rows, long long cols) {
    static const RowShape many[] = {{16, 4},  {16, 8},  {16, 12},  {16, 16},  {32, 12},  {64, 8},    {64, 12},  {64, 16},
                                    {256, 8}, {256, 12}, {256, 16}, {512, 12}, {512, 16}, {1024, 12}, {1024, 16}};
    static const RowShape few[] = {{64, 4},    {64, 8},   {64, 12},  {64, 16},   {256, 8},  {256, 12},
                                   {256, 16}, {512, 12}, {512, 16}, {1024, 12}, {1024, 16}};
    const RowShape s = rows >= NORM_FEW ? first_fit(many, sizeof many / sizeof *many, cols)
                                        : first_fit(few, sizeof few / sizeof *few, cols);
    const long long rpb = s.t > 64 ? 1 : grad_block(s.t) / s.t, want = (rows + rpb - 1) / rpb;
    const long long cap = s.t == 256 && rows > 8 * NCU ? 2 * NCU : NCU;
    return NormPlan{s.t, s.e, (int)(want < 1 ? 1 : want > cap ? cap : want)};
}

int n_tops(long long rows, int e_row) {
    if (!e_row || rows <= TOPS_ROWS) return 0;
    const long long n = (rows + TOPS_ROWS - 1) / TOPS_ROWS;
    return (int)(n > TOPS_MAX ? TOPS_MAX : n);
}

// The smallest t * e that holds a row, e a multiple of the eight elements
// that share a block of random bits, on as many blocks as are resident (16384 x
// 1024 into a whole-tensor result in 512, 1536 and 4096 blocks: 21.5, 20.5, 28.4
// us; 8192 x 2048 with a residual: 29.2, 18.5, 18.5).
NormPlan dropout_plan(long long rows, long long cols) {
    const int ts[] = {8, 16, 32, 64, 256, 1024};
    NormPlan p{1024, 0, 1};
    for (int t : ts)
        for (int e = t == 16 || t == 32 || t == 64 ? 16 : 8; e <= (t == 1024 ? 16 : 24); e += 8)
            if (cols <= (long long)t * e && (p.e == 0 || t * e < p.t * p.e)) p = NormPlan{t, e, 1};
    const long long rpb = p.t > 256 ? 1 : 256 / p.t;
    const long long want = (rows + rpb - 1) / rpb, cap = p.t > 256 ? 2 * NCU : 6 * NCU;
    p.grid = (int)(want < 1 ? 1 : want > cap ? cap : want);
    return p;
}

// Row chunks of whole trips (64 rows), about four blocks a CU, but no shorter
// than two trips unless that leaves CUs idle (25216 x 2304 in chunks of 128,
// 256 and 512: 20.6, 19.5, 23.3 us; 8192 x 1024 in 64, 128, 256: 8.0, 7.9, 9.7;
// 1000 x 1000 in 64 and 128: 7.9, 9.8).
ColPlan col_plan(long long rows, long long cols) {
    const long long gx = (cols + 255) / 256;
    long long trips = (rows * gx + 256 * NCU - 1) / (256 * NCU);
    if (trips < 2) trips = rows * gx > 64 * NCU ? 2 : 1;
    if (trips > 1 << 17) trips = 1 << 17;  // 2^23 rows: 32-bit sums
    const long long chunk = trips * 64;
    return ColPlan{rows > chunk ? (int)((rows + chunk - 1) / chunk) : 1, (int)chunk};
}

static ColWs carve_cols(Carve &c, long long parts, long long cols, bool wide) {
    ColWs w{};
    const size_t n = (size_t)(cols > 0 ? cols : 1), np = (size_t)col_pitch((int)n);
    w.top = c.take<int>(1);
    w.tops = c.take<int>(TOPS_MAX);
    if (wide) w.p64 = c.take<long long>((size_t)parts * np);
    w.p32 = c.take<int>((size_t)parts * np);
    w.sums = c.take<long long>(2 * n);
    w.need = c.take<int>(2 * ((n + 15) / 16));
    return w;
}

NormWs carve_norm_fwd(Carve &c, long long rows, long long cols) {
    NormWs w{};
    w.bmax = c.take<int>((size_t)norm_fwd_plan(rows, cols).grid);
    w.stat = c.take<char>((size_t)rows * 16);
    return w;
}

NormWs carve_norm_bwd(Carve &c, long long rows, long long cols) {
    NormWs w{};
    const NormPlan p = norm_bwd_plan(rows, cols);
    w.bmax = c.take<int>((size_t)p.grid);
    w.stat = c.take<char>((size_t)rows * 32);
    w.c = carve_cols(c, p.grid, cols, true);
    return w;
}

ColWs carve_linear_db(Carve &c, long long rows, long long cols) {
    return carve_cols(c, col_plan(rows, cols).parts, cols, false);
}

int *carve_dropout(Carve &c, long long rows, long long cols) {
    return c.take<int>((size_t)dropout_plan(rows, cols).grid);
}

AttFwdWs carve_attention_fwd(Carve &c, long long rows, long long heads, long long kv, long long d) {
    AttFwdWs w;
    w.v16 = c.take<int16_t>((size_t)(rows * heads * d));
    w.p16 = c.take<int16_t>((size_t)(rows * heads));
    w.xp = c.take<int8_t>((size_t)(rows * (heads + 2 * kv) * r16(d)));
    return w;
}

size_t attention_fwd_ws(long long rows, long long heads, long long kv, long long d) {
    Carve c{nullptr, HEADER};
    carve_attention_fwd(c, rows, heads, kv, d);
    return align256(c.off);
}

AttBwdWs carve_attention_bwd(Carve &c, long long rows, long long heads, long long kv, long long d) {
    AttBwdWs w;
    w.v16 = c.take<int16_t>((size_t)(rows * (heads + 2 * kv) * d));
    w.p16 = c.take<int16_t>((size_t)(rows * (heads + 2 * kv)));
    w.dots = c.take<char>((size_t)(rows * heads * 8));
    w.norm = c.take<int8_t>((size_t)(rows * kv));
    w.row = c.take<char>((size_t)(rows * heads * 32));
    w.key = c.take<char>((size_t)(rows * kv * 4));
    w.xp = c.take<int8_t>((size_t)(rows * (heads + 2 * kv) * r16(d)));
    w.dyp = c.take<int8_t>((size_t)(rows * heads * r16(d)));
    return w;
}

size_t attention_bwd_ws(long long rows, long long heads, long long kv, long long d) {
    Carve c{nullptr, HEADER};
    carve_attention_bwd(c, rows, heads, kv, d);
    return align256(c.off);
}

RopePlan rope_plan(long long rows, long long cols, bool eight, bool whole) {
    RopePlan p{256, 0, 1};
    if (eight) {
        const long long units = cols / 8;
#define IE_TRY_(T_, N_)                                                                       \
    if (units <= (long long)T_ * N_ && (p.nu == 0 || T_ * N_ < p.t * p.nu)) p = RopePlan{T_, N_, 1};
        IE_ROPE_SHAPES(IE_TRY_)
#undef IE_TRY_
    }
    const long long rpb = p.nu ? 256 / p.t : 1, want = (rows + rpb - 1) / rpb;
    const int most = whole ? ROPE_BLOCKS : 8 * ROPE_BLOCKS;
    p.grid = (int)(want < 1 ? 1 : want > most ? most : want);
    return p;
}

int *carve_rope(Carve &c, long long, long long) { return c.take<int>(ROPE_BLOCKS); }

size_t rope_ws(long long rows, long long cols) {
    Carve c{nullptr, HEADER};
    carve_rope(c, rows, cols);
    return align256(c.off);
}

CacheWs carve_attention_cache(Carve &c, long long n, long long tokens, long long heads, long long d) {
    const size_t blocks = (size_t)((tokens + CACHE_BLOCK - 1) / CACHE_BLOCK);
    CacheWs w;
    w.num = c.take<int>((size_t)n * blocks * (size_t)(heads * d));
    w.top = c.take<char>((size_t)n * blocks * (size_t)heads * 16);
    w.v16 = c.take<int16_t>((size_t)n * (size_t)(heads * d));
    w.p16 = c.take<int16_t>((size_t)n * (size_t)(heads * d / 16));  // a need for 16 elements at least
    return w;
}

size_t attention_cache_ws(long long n, long long tokens, long long heads, long long d) {
    Carve c{nullptr, HEADER};
    carve_attention_cache(c, n, tokens, heads, d);
    return align256(c.off);
}

ie_status check_cache(const ie_cache *c) {
    if (!c) return IE_ERR_NULL;
    if (c->pages < 0 || c->page < 1 || c->kv_heads < 1 || c->head_dim < 1) return IE_ERR_SHAPE;
    if (c->pages > 0 && (!c->k || !c->v || !c->k_exp || !c->v_exp)) return IE_ERR_NULL;
    if ((c->page & (c->page - 1)) || c->head_dim % 16 || c->head_dim > ATT_HEAD_MAX ||
        (long long)c->pages * c->page > DIM_MAX || c->kv_heads > (1 << 16))
        return IE_ERR_UNSUPPORTED;
    if (((uintptr_t)c->k | (uintptr_t)c->v) % 8) return IE_ERR_UNSUPPORTED;
    return IE_OK;
}

// The heads of an attention call and the matrix that holds them.
ie_status check_attention(const ie_attention_desc *d, const ie_mat *X, long long cols) {
    if (!d) return IE_ERR_NULL;
    const ie_status s = check_mat(X);
    if (s != IE_OK) return s;
    if (d->heads < 1 || d->kv_heads < 1 || d->head_dim < 1 || d->heads % d->kv_heads || d->n_seq < 0)
        return IE_ERR_SHAPE;
    if (X->cols != cols) return IE_ERR_SHAPE;
    if (!d->offsets != !d->n_seq) return IE_ERR_SHAPE;
    if (d->head_dim > ATT_HEAD_MAX || (uintptr_t)d->offsets % 4) return IE_ERR_UNSUPPORTED;
    // 64 rows of a tile within a 32-bit window
    if (((long long)d->heads + 2ll * d->kv_heads) * r16(d->head_dim) > ATT_COLS_MAX) return IE_ERR_UNSUPPORTED;
    // 2^-30 .. 2^30: r = scale log2(e) 2^e keeps clear of fp32's ends (a NaN is refused too)
    if (!(d->scale >= 0x1p-30f && d->scale <= 0x1p30f)) return IE_ERR_UNSUPPORTED;
    // tiles of 32 rows and up (those of 16 are few, see ie_attention_bwd.hip), 4 rows a workgroup in the rounding
    if ((att_slots(X->rows, d->n_seq, 32) + 8) * d->heads > ATT_BLOCKS_MAX || X->rows > 4 * ATT_BLOCKS_MAX)
        return IE_ERR_UNSUPPORTED;
    return IE_OK;
}

size_t dropout_ws(long long rows, long long cols) {
    Carve c{nullptr, HEADER};
    carve_dropout(c, rows, cols);
    return align256(c.off);
}

size_t norm_fwd_ws(long long rows, long long cols) {
    Carve c{nullptr, HEADER};
    carve_norm_fwd(c, rows, cols);
    return align256(c.off);
}

size_t norm_bwd_ws(long long rows, long long cols) {
    Carve c{nullptr, HEADER};
    carve_norm_bwd(c, rows, cols);
    return align256(c.off);
}

size_t linear_db_ws(long long rows, long long cols) {
    Carve c{nullptr, HEADER};
    carve_linear_db(c, rows, cols);
    return align256(c.off);
}

size_t linear_fwd_ws(long long M, long long N, long long K, const Force &f) {
    Carve c{nullptr, HEADER};
    carve_linear_fwd(c, M, N, K, f);
    return align256(c.off);
}

// Also enough for the plain product, which runs when there is neither bias
// nor residual.
size_t linear_fused_ws(long long M, long long N, long long K, const Force &f) {
    Carve c{nullptr, HEADER};
    carve_linear_fused(c, M, N, K, f);
    return mx(align256(c.off), linear_fwd_ws(M, N, K, f));
}

size_t linear_dx_ws(long long M, long long N, long long K, const Force &f) {
    Carve c{nullptr, HEADER};
    carve_linear_dx(c, M, N, K, f);
    return align256(c.off);
}

size_t linear_dw_ws(long long M, long long N, long long K, const Force &fw) {
    Carve c{nullptr, HEADER};
    carve_linear_dw(c, M, N, K, fw);
    return align256(c.off);
}

size_t conv_fwd_ws(const ConvGeom &g, const Force &f) {
    Carve c{nullptr, HEADER};
    carve_conv_fwd(c, g, f);
    return align256(c.off);
}

size_t conv_bwd_ws(const ConvGeom &g, const Force &f, const Force &fw) {
    Carve c{nullptr, HEADER};
    carve_conv_bwd(c, g, f, fw);
    return align256(c.off);
}

size_t bmm_ws(long long Z, long long M, long long N, long long K) {
    size_t best = HEADER;
    for (int form = 0; form < 3; ++form) {
        Carve c{nullptr, HEADER};
        carve_bmm(c, form, Z, M, N, K);
        best = mx(best, align256(c.off));
    }
    return best;
}

}  // namespace ie
