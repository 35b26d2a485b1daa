// Host-only check of the launches of the block operators (tests/test_plan_launch.py):
// a launch has fewer than 2^32 threads along an axis, whatever the shape.
// Exit status 0 when every check passes.
#include <stdio.h>
#include <stdlib.h>

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

int main() {
    for (long long e = 0; e <= 30; ++e)
        for (long long d = -17; d <= 17; ++d) {
            const long long c = (1ll << e) + d;
            if (c >= 1 && c <= LONG_COLS_MAX) check_columns(c);
        }
    printf("plan_launch_check: %lld checks\n", g_checks);
    return 0;
}
