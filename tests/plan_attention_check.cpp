// Host-side checks of the attention, rotary and cache entry points' plans
// (built with the address and undefined-behaviour sanitizers): every workspace
// is allocated at the size its query returns and each buffer's last byte, as
// the kernels index it, is touched; tile slots cover every row of every
// sequence once; every rotary plan has a kernel that holds its rows.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../integer_only_dnn_amd/csrc/ie_plan.h"

using namespace ie;

static long checks = 0;
#define CHECK(x)                                                        \
    do {                                                                \
        ++checks;                                                       \
        if (!(x)) {                                                     \
            std::printf("FAILED %s line %d\n", #x, __LINE__);           \
            std::exit(1);                                               \
        }                                                               \
    } while (0)

template <class T>
static void touch(T *p, size_t n) {
    if (!n) return;
    p[0] = T{};
    p[n - 1] = T{};
    CHECK((uintptr_t)p % 256 == 0);
}

static void workspaces() {
    const long long rows_[] = {0, 1, 7, 64, 129, 1000}, d_[] = {1, 7, 32, 64, 100, 128};
    const int heads_[][2] = {{1, 1}, {4, 2}, {12, 12}, {17, 1}};
    for (long long rows : rows_)
        for (auto &hk : heads_)
            for (long long d : d_) {
                const long long h = hk[0], kv = hk[1];
                {
                    std::vector<char> b(attention_fwd_ws(rows, h, kv, d) + 256);
                    char *base = (char *)(((uintptr_t)b.data() + 255) & ~(uintptr_t)255);
                    Carve c{base, HEADER};
                    const AttFwdWs w = carve_attention_fwd(c, rows, h, kv, d);
                    touch(w.v16, rows * h * d);
                    touch(w.p16, rows * h);
                    touch(w.xp, rows * (h + 2 * kv) * ((d + 15) / 16 * 16));
                    CHECK(align256(c.off) == attention_fwd_ws(rows, h, kv, d));
                }
                {
                    std::vector<char> b(attention_bwd_ws(rows, h, kv, d) + 256);
                    char *base = (char *)(((uintptr_t)b.data() + 255) & ~(uintptr_t)255);
                    Carve c{base, HEADER};
                    const AttBwdWs w = carve_attention_bwd(c, rows, h, kv, d);
                    touch(w.v16, rows * (h + 2 * kv) * d);
                    touch(w.p16, rows * (h + 2 * kv));
                    touch((char *)w.dots, rows * h * 8);
                    touch(w.norm, rows * kv);
                    touch((char *)w.row, rows * h * 32);
                    touch((char *)w.key, rows * kv * 4);
                    touch(w.xp, rows * (h + 2 * kv) * ((d + 15) / 16 * 16));
                    touch(w.dyp, rows * h * ((d + 15) / 16 * 16));
                    CHECK(align256(c.off) == attention_bwd_ws(rows, h, kv, d));
                }
                for (long long tokens : {0ll, 1ll, 255ll, 256ll, 257ll, 5000ll}) {
                    if (rows * tokens > 300000) continue;
                    std::vector<char> b(attention_cache_ws(rows, tokens, h, d) + 256);
                    char *base = (char *)(((uintptr_t)b.data() + 255) & ~(uintptr_t)255);
                    Carve c{base, HEADER};
                    const CacheWs w = carve_attention_cache(c, rows, tokens, h, d);
                    const long long blocks = (tokens + CACHE_BLOCK - 1) / CACHE_BLOCK;
                    touch(w.num, rows * blocks * h * d);
                    touch((char *)w.top, rows * blocks * h * 16);
                    touch(w.v16, rows * h * d);
                    touch(w.p16, rows * (h * d / 16));
                    CHECK(align256(c.off) == attention_cache_ws(rows, tokens, h, d));
                }
            }
}

// The kernels' way from a slot to its sequence's tile.
static void slots() {
    unsigned seed = 1;
    auto next = [&](unsigned m) {
        seed = seed * 1664525u + 1013904223u;
        return (seed >> 8) % m;
    };
    for (int turn = 0; turn < 400; ++turn) {
        const int n = 1 + (int)next(40), bm = turn % 2 ? 128 : 64;
        std::vector<int> off(n + 1);
        off[0] = (int)next(300);
        for (int s = 0; s < n; ++s) off[s + 1] = off[s] + (next(3) ? (int)next(500) : 0);
        const int rows = off[n] + (int)next(200);
        std::vector<int> seen(rows, 0);
        const int total = (int)att_slots(rows, n, bm);
        for (int slot = 0; slot < total; ++slot) {
            int lo = 0, hi = n - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (off[mid] / bm + mid <= slot) lo = mid;
                else hi = mid - 1;
            }
            const int len = off[lo + 1] - off[lo], at = slot - (off[lo] / bm + lo);
            const int first = at < 0 || at > len / bm ? len : at * bm;
            for (int r = first; r < len && r < first + bm; ++r) ++seen[off[lo] + r];
        }
        for (int r = 0; r < rows; ++r) CHECK(seen[r] == (r >= off[0] && r < off[n] ? 1 : 0));
    }
    CHECK(att_slots(1000, 0, 128) * 128 >= 1000 && att_slots(1024, 0, 128) * 128 >= 1024);
}

static void rope() {
    for (long long cols = 8; cols <= 20000; cols += 8)
        for (long long rows : {1ll, 5ll, 100ll, 100000ll}) {
            const RopePlan p = rope_plan(rows, cols, true);
            bool built = p.nu == 0;
#define IE_IS(T_, N_) built |= p.t == T_ && p.nu == N_;
            IE_ROPE_SHAPES(IE_IS)
#undef IE_IS
            CHECK(built);
            CHECK(p.nu == 0 ? cols > 16384 : (long long)p.t * p.nu * 8 >= cols);
            CHECK(p.grid >= 1 && p.grid <= ROPE_BLOCKS && rope_plan(rows, cols, true, false).grid >= p.grid);
            const RopePlan any = rope_plan(rows, cols, false);
            CHECK(any.nu == 0 && any.grid >= 1 && any.grid <= ROPE_BLOCKS);
        }
    std::vector<char> b(rope_ws(10, 10) + 256);
    char *base = (char *)(((uintptr_t)b.data() + 255) & ~(uintptr_t)255);
    Carve c{base, HEADER};
    touch(carve_rope(c, 10, 10), ROPE_BLOCKS);
}

int main() {
    workspaces();
    slots();
    rope();
    std::printf("plan_attention_check: %ld checks\n", checks);
    return 0;
}
