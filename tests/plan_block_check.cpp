// Host-only check of the plans and workspace layouts of the layer norm, column
// sum, dropout and bias / residual product entry points, built with address
// and undefined-behaviour sanitizers (tests/test_plan_block.py): over shapes on
// and beside every edge, a plan holds its rows, its launches stay within their
// limits, and what the kernels index lies inside the workspace the size query
// asks for, no buffer over another.  Exit status 0 when every check passes.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "../integer_only_dnn_amd/csrc/ie_plan.h"

using namespace ie;

static long long g_checks = 0;

#define REQUIRE(cond, ...)                                                    \
    do {                                                                      \
        ++g_checks;                                                           \
        if (!(cond)) {                                                        \
            fprintf(stderr, "FAIL %s:%d: %s\n  ", __FILE__, __LINE__, #cond); \
            fprintf(stderr, __VA_ARGS__);                                     \
            fprintf(stderr, "\n");                                            \
            exit(1);                                                          \
        }                                                                     \
    } while (0)

// The workspace as addresses only: nothing is allocated.
struct Layout {
    char *base = (char *)(1ull << 40);
    std::vector<std::pair<size_t, size_t>> used;  // first byte, bytes
    template <class T>
    void use(const T *p, size_t count) {
        if (!count) return;
        REQUIRE(p != nullptr, "a buffer of %zu is missing", count);
        used.push_back({(size_t)((const char *)p - base), count * sizeof(T)});
    }
    void check(size_t bytes, const char *what, long long a, long long b, long long c) {
        std::sort(used.begin(), used.end());
        size_t end = HEADER;
        for (auto &u : used) {
            REQUIRE(u.first >= end, "%s %lld %lld %lld: buffers overlap", what, a, b, c);
            end = u.first + u.second;
        }
        REQUIRE(end <= bytes, "%s %lld %lld %lld: %zu bytes of %zu", what, a, b, c, end, bytes);
    }
};

static void use_cols(Layout &l, const ColWs &w, long long parts, long long cols, bool wide) {
    l.use(w.top, 1);
    l.use(w.tops, TOPS_MAX);
    if (wide) l.use(w.p64, (size_t)parts * col_pitch((int)cols));
    l.use(w.p32, (size_t)parts * col_pitch((int)cols));
    l.use(w.sums, 2 * (size_t)cols);
    l.use(w.need, 2 * (size_t)((cols + 15) / 16));
}

static void check_rows(long long rows, long long cols) {
    if (cols <= NORM_COLS_MAX) {
        const NormPlan f = norm_fwd_plan(rows, cols), b = norm_bwd_plan(rows, cols), o = norm_one_plan(rows, cols);
        REQUIRE((long long)f.t * f.e >= cols && f.e % 4 == 0 && f.grid >= 1, "forward %lld x %lld", rows, cols);
        REQUIRE((long long)b.t * b.e >= cols && b.e % 4 == 0 && b.grid >= 1, "backward %lld x %lld", rows, cols);
        if (o.grid)
            REQUIRE((long long)o.t * o.e >= cols && rows * o.t <= 1024 && o.grid == 1, "one %lld x %lld", rows, cols);
        // a backward result that one block holds is that block's only trip
        if (b.grid == 1 && b.t <= 64) REQUIRE(rows * b.t <= grad_block(b.t), "backward %lld x %lld", rows, cols);
        Layout l;
        Carve c{l.base, HEADER};
        const NormWs w = carve_norm_fwd(c, rows, cols);
        l.use(w.bmax, f.grid);
        l.use((char *)w.stat, (size_t)rows * 16);
        l.check(norm_fwd_ws(rows, cols), "norm fwd", rows, cols, 0);
        Layout m;
        Carve d{m.base, HEADER};
        const NormWs v = carve_norm_bwd(d, rows, cols);
        m.use(v.bmax, b.grid);
        m.use((char *)v.stat, (size_t)rows * 32);
        use_cols(m, v.c, b.grid, cols, true);
        m.check(norm_bwd_ws(rows, cols), "norm bwd", rows, cols, 0);
    }
    const NormPlan d = dropout_plan(rows, cols);
    REQUIRE(d.grid >= 1 && (d.e == 0 ? cols > 16384 : d.e % 8 == 0 && (long long)d.t * d.e >= cols), "dropout %lld x %lld",
            rows, cols);
    Layout l;
    Carve c{l.base, HEADER};
    l.use(carve_dropout(c, rows, cols), d.grid);
    l.check(dropout_ws(rows, cols), "dropout", rows, cols, 0);
    const ColPlan p = col_plan(rows, cols);
    REQUIRE(p.parts >= 1 && p.parts <= 65535 && p.chunk >= 1 && p.chunk <= 1 << 23, "chunks %lld x %lld", rows, cols);
    REQUIRE((long long)p.parts * p.chunk >= rows && (rows == 0 || (long long)(p.parts - 1) * p.chunk < rows),
            "chunks %lld x %lld: %d of %d", rows, cols, p.parts, p.chunk);
    for (int e_row = 0; e_row < 2; ++e_row) REQUIRE(n_tops(rows, e_row) <= TOPS_MAX, "tops %lld", rows);
    Layout m;
    Carve k{m.base, HEADER};
    use_cols(m, carve_linear_db(k, rows, cols), p.parts, cols, false);
    m.check(linear_db_ws(rows, cols), "column sums", rows, cols, 0);
}

static void check_product(long long M, long long N, long long K) {
    const Force none{0, 0, 0, -1, 1};
    const long long Kp = (K + 15) / 16 * 16, Np = (N + 15) / 16 * 16;
    for (int rg = 0; rg < 2; ++rg) {
        Layout l;
        Carve c{l.base, HEADER};
        const LinearFusedWs w = carve_linear_fused(c, M, N, K, none);
        const int ni = rows_plan(M, N, Kp, rg, none);
        if (few_plan(M, N, Kp, none)) {
            REQUIRE(!ni && M <= FEW_ROWS, "%lld %lld %lld", M, N, K);
            l.use(w.few_acc, (size_t)(M * Np));
            l.use(w.few_w, (size_t)(M * Np / 16));
        } else if (ni) {
            REQUIRE(rg && ni <= 4 && 256ll * ni >= N && M * K >= 16 && N >= 16, "%lld %lld %lld", M, N, K);
            REQUIRE(rows_steps(K) % 2 == 0 && rows_steps(K) * 32ll >= K, "%lld", K);
            // every wave's share of the weight is inside a 31-bit window
            REQUIRE(rows_weight(ni, K) <= rows_weight(ni, Kp) && rows_weight(ni, Kp) < 1ull << 31, "%lld %lld", N, K);
            l.use(w.wt, rows_weight(ni, K));
        } else {
            const Plan p = plan_add(M, N, Kp, rg, none);
            REQUIRE(plan_valid(p, M, N, Kp, rg, FAM_ADD), "%lld %lld %lld", M, N, K);
            if (Kp != K) {
                l.use(w.l.xp, (size_t)(M * Kp));
                l.use(w.l.wp, (size_t)(N * Kp));
            }
            const long long tm = (M + p.t.bm() - 1) / p.t.bm(), tn = (N + p.t.bn() - 1) / p.t.bn();
            if (p.mode == PLAN_RTO) {
                l.use(w.l.pw.v16, (size_t)(M * add_pitch((int)N)));
                l.use(w.l.pw.p16, (size_t)(rg ? M * tn : tm * tn));
            } else if (p.mode == PLAN_SPLIT) {
                l.use(w.l.pw.partial, (size_t)p.splits * M * N);
                l.use(w.bmax, SPLIT_ADD_BLOCKS);
            }
        }
        l.check(linear_fused_ws(M, N, K, none), "product", M, N, K);
    }
}

int main() {
    const long long rows[] = {1, 2, 8, 9, 16, 17, 33, 64, 65, 127, 1000, 2047, 2048, 4095, 4096, 16384, 16385, 25216,
                              65536, 65537, 131072, 1000003, 1ll << 24, 1ll << 27};
    const long long cols[] = {1, 3, 4, 5, 63, 64, 65, 129, 192, 256, 257, 384, 385, 512, 513, 768, 769, 1024, 1025, 2048,
                              4096, 4097, 6144, 6145, 8192, 8193, 12289, 16384, 16385, 24577, 100000, 1 << 20};
    for (long long r : rows)
        for (long long c : cols)
            if (r * c <= 1ll << 34) check_rows(r, c);
    check_rows(1, 1ll << 30);
    check_rows(1ll << 31, 1);
    const long long ms[] = {1, 5, 16, 17, 64, 65, 100, 128, 129, 700, 2047, 2048, 2049, 6143, 6144, 20000, 50432, 1 << 20};
    const long long ns[] = {1, 3, 16, 63, 64, 65, 128, 129, 200, 256, 257, 512, 513, 768, 1000, 1024, 1025, 2304, 4099, 32000};
    const long long ks[] = {1, 15, 16, 17, 96, 256, 257, 768, 1024, 1040, 2048, 2049, 4096, 16384, 65536};
    for (long long m : ms)
        for (long long n : ns)
            for (long long k : ks)
                if (m * n <= 1ll << 31 && m * k <= 1ll << 32) check_product(m, n, k);
    printf("plan_block_check: %lld checks\n", g_checks);
    return 0;
}
