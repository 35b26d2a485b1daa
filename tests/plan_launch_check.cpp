// Host-only check of the launches of the block operators (tests/test_plan_launch.py):
// a launch has fewer than 2^32 threads along an axis, whatever the shape; every
// split of rows over threads that is planned is built, and every one that is
// built is planned for some shape.  With arguments KIND ROWS COLS ROWS COLS ...
// (KIND forward, backward or dropout) it checks that those shapes take every
// split whose blocks can take rows in turn to a second trip at least.  Exit
// status 0 when every check passes.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <set>
#include <utility>

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

// Column sums: a block of 1024 threads closes 16 columns at a time.
static void check_columns(long long cols) {
    const long long nb = col_blocks(cols);
    REQUIRE(nb >= 1 && nb * 16 >= (cols < 16 * COL_BLOCKS ? cols : 16 * COL_BLOCKS), "%lld columns: %lld blocks", cols, nb);
    REQUIRE((nb - 1) * 16 < cols, "%lld columns: %lld blocks", cols, nb);
    REQUIRE(nb * 1024 < 1ll << 32, "%lld columns: %lld blocks", cols, nb);
    REQUIRE((cols + 255) / 256 * 256 < 1ll << 32, "%lld columns", cols);
}

// The splits planned for rows of each length, over few rows and many.
using Splits = std::set<std::pair<int, int>>;

static void check_splits() {
    Splits fwd, one, bwd, drop;
    for (long long rows : {1ll, 15ll, 16ll, 17ll, 63ll, 64ll, 65ll, 1000ll, NORM_FEW - 1, NORM_FEW, NORM_FEW + 1, 1000000ll})
        for (long long cols = 1; cols <= 30000; ++cols) {
            const NormPlan d = dropout_plan(rows, cols);
            REQUIRE(dropout_built(d), "dropout %lld x %lld: (%d, %d)", rows, cols, d.t, d.e);
            drop.insert({d.t, d.e});
            if (cols > NORM_COLS_MAX) continue;
            const NormPlan f = norm_fwd_plan(rows, cols), o = norm_one_plan(rows, cols), b = norm_bwd_plan(rows, cols);
            REQUIRE(norm_fwd_built(f), "forward %lld x %lld: (%d, %d)", rows, cols, f.t, f.e);
            REQUIRE(norm_bwd_built(b), "backward %lld x %lld: (%d, %d)", rows, cols, b.t, b.e);
            REQUIRE(!o.grid || norm_one_built(o), "one block %lld x %lld: (%d, %d)", rows, cols, o.t, o.e);
            fwd.insert({f.t, f.e});
            bwd.insert({b.t, b.e});
            if (o.grid) one.insert({o.t, o.e});
        }
#define IE_PLANNED(T_, E_) REQUIRE(planned.count({T_, E_}), "(%d, %d) is built and never planned", T_, E_);
    {
        const Splits &planned = fwd;
        IE_NORM_FWD(IE_PLANNED)
    }
    {
        const Splits &planned = one;
        IE_NORM_ONE(IE_PLANNED)
    }
    {
        const Splits &planned = bwd;
        IE_NORM_BWD(IE_PLANNED)
    }
    {
        const Splits &planned = drop;
        IE_DROP_SHAPES(IE_PLANNED)
    }
#undef IE_PLANNED
    const NormPlan none{7, 4, 1};
    REQUIRE(!norm_fwd_built(none) && !norm_one_built(none) && !norm_bwd_built(none) && !dropout_built(none), "(7, 4)");
}

// A block's threads (backward, dropout and forward differ in them) and its trips.
static long long trips(const char *kind, long long rows, long long cols, NormPlan &p) {
    long long block = 0;
    if (!strcmp(kind, "forward")) p = norm_fwd_plan(rows, cols), block = p.t > 256 ? p.t : 256;
    if (!strcmp(kind, "backward")) p = norm_bwd_plan(rows, cols), block = grad_block(p.t);
    if (!strcmp(kind, "dropout")) p = dropout_plan(rows, cols), block = p.t > 256 ? p.t : 256;
    REQUIRE(block, "%s", kind);
    const long long each = block / p.t * p.grid;
    return (rows + each - 1) / each;
}

static void check_trips(const char *kind, int n, char **size) {
    Splits can, done;
    NormPlan p;
    const long long longest = strcmp(kind, "dropout") ? NORM_COLS_MAX : 30000;
    for (long long rows : {NORM_FEW - 1, 1000000ll})
        for (long long cols = 1; cols <= longest; ++cols)
            if (trips(kind, rows, cols, p) > 1) can.insert({p.t, p.e});
    for (int i = 0; i + 1 < n; i += 2)
        if (trips(kind, atoll(size[i]), atoll(size[i + 1]), p) > 1) done.insert({p.t, p.e});
    REQUIRE(!can.empty(), "%s", kind);
    for (const auto &c : can) REQUIRE(done.count(c), "%s: no shape takes (%d, %d) to a second trip", kind, c.first, c.second);
}

int main(int argc, char **argv) {
    if (argc > 1) {
        check_trips(argv[1], argc - 2, argv + 2);
        printf("plan_launch_check: %lld checks\n", g_checks);
        return 0;
    }
    check_splits();
    for (long long e = 0; e <= 30; ++e)
        for (long long d = -17; d <= 17; ++d) {
            const long long c = (1ll << e) + d;
            if (c >= 1 && c <= LONG_COLS_MAX) check_columns(c);
        }
    printf("plan_launch_check: %lld checks\n", g_checks);
    return 0;
}
