// A host check of which tile of which sequence, and which head, a workgroup of
// attention takes (csrc/ie_attn_index.h, the kernels' own code), with the 64
// lanes of a wave written out: every tile of every sequence and every head is met exactly
// once, whatever the lengths, tile heights, numbers of sequences and launch orders.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../integer_only_dnn_amd/csrc/ie_attn_index.h"

using namespace ie;

static long checks = 0;
#define CHECK(x)                                                           \
    do {                                                                   \
        ++checks;                                                          \
        if (!(x)) {                                                        \
            std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x);            \
            std::exit(1);                                                  \
        }                                                                  \
    } while (0)

struct Lanes64 {
    struct Int {
        int v[64];
    };
    template <class F>
    Int each(F f) const {
        Int r;
        for (int l = 0; l < 64; ++l) r.v[l] = f(l);
        return r;
    }
    template <class F>
    uint64_t ballot(F f) const {
        uint64_t r = 0;
        for (int l = 0; l < 64; ++l) r |= (uint64_t)(f(l) ? 1 : 0) << l;
        return r;
    }
    int of(const Int &x, int lane) const { return x.v[lane]; }
    int at(const Int &x, int lane) const { return x.v[lane]; }
    int sum(const Int &x) const {
        int r = 0;
        for (int v : x.v) r += v;
        return r;
    }
    int max(const Int &x) const {
        int r = x.v[0];
        for (int v : x.v) r = v > r ? v : r;
        return r;
    }
};

// What the functions read of a call, with bounds.
struct Off {
    const std::vector<int> *v = nullptr;
    int operator[](int i) const {
        CHECK(i >= 0 && i < (int)v->size());
        return (*v)[i];
    }
    explicit operator bool() const { return v != nullptr; }
    bool operator!() const { return v == nullptr; }
};
struct Call {
    Off off;
    long long rows;
    int n_seq, most, kv, chunk;
};

static unsigned seed = 1;
static int next(unsigned m) {
    seed = seed * 1664525u + 1013904223u;
    return (int)((seed >> 8) % m);
}

// All workgroups of a launch; `most`: rows of a sequence that are taken at most.
template <bool HEAVY>
static void launch(const std::vector<int> *off, long long rows, int bm, int kv, int per, bool alike, int most) {
    const int n = off ? (int)off->size() - 1 : 0;
    Call p{Off{off}, rows, n, most, kv, 0};
    p.chunk = att_chunk(rows, n, kv, bm, alike && off);
    std::vector<int> start, len;
    for (int s = 0; s < (off ? n : 1); ++s) {
        const Span x = off ? span_of(p, (*off)[s], (*off)[s + 1]) : Span{0, (int)(rows < most ? rows : most)};
        start.push_back(x.a);
        len.push_back(x.n);
    }
    // tiles by their first row, heads apart
    const long long slots = att_slots(rows, n, bm);
    const unsigned grid = att_grid(slots, kv, per);
    std::vector<unsigned char> seen((size_t)rows * kv * per, 0);
    int before = 1 << 30;
    long tiles = 0;
    for (unsigned block = 0; block < grid; ++block) {
        const Item it = att_item(p, per, (int)block, (int)grid);
        CHECK(it.rank >= 0 && it.kvh >= 0 && it.kvh < kv && it.gh >= 0 && it.gh < per);
        Span sp;
        int tile;
        if (!rank_tile<HEAVY>(Lanes64{}, p, it.rank, bm, sp, tile)) continue;
        CHECK(tile >= 0 && (long long)tile * bm < sp.n && sp.a >= 0 && sp.a + sp.n <= rows);
        unsigned char &x = seen[((size_t)(sp.a + tile * bm) * kv + it.kvh) * per + it.gh];
        CHECK(!x);
        x = 1;
        ++tiles;
        if (HEAVY && off && n <= 64 && kv == 1 && per == 1) {  // in the order of their work
            CHECK(tile <= before);
            before = tile;
        }
    }
    long want = 0;
    for (size_t s = 0; s < start.size(); ++s)
        for (int t = 0; t * bm < len[s]; ++t)
            for (int h = 0; h < kv * per; ++h) {
                CHECK(seen[(size_t)(start[s] + t * bm) * kv * per + h]);
                ++want;
            }
    CHECK(tiles == want);
}

static std::vector<int> offsets(int n, int longest, int empty) {
    std::vector<int> off{next(300)};
    for (int s = 0; s < n; ++s) off.push_back(off.back() + (next(10) < empty ? 0 : 1 + next(longest)));
    return off;
}

static void both(const std::vector<int> *off, long long rows, int bm, int kv, int per, bool alike, int most = 131071) {
    launch<false>(off, rows, bm, kv, per, alike, most);
    launch<true>(off, rows, bm, kv, per, false, most);
}

int main(int argc, char **argv) {
    const bool large = argc > 1;  // (the largest numbers of sequences, without sanitizers)
    const int heights[] = {16, 32, 64, 256};
    for (int bm : heights) {
        for (long long rows : {1ll, 15ll, 16ll, 17ll, 1000ll, 5000ll}) both(nullptr, rows, bm, 1 + next(3), 1 + next(3), true);
        for (int n : {1, 2, 5, 63, 64, 65, 100, 700}) {
            for (int turn = 0; turn < (n < 100 ? 12 : 3); ++turn) {
                const int longest[] = {3, 40, 300, 2000};
                const auto off = offsets(n, longest[turn % 4], turn % 3 == 2 ? 9 : 3 * (turn % 3));
                if (off.back() > 60000) continue;
                both(&off, off.back() + 1 + next(200), bm, 1 + next(3), 1 + next(3), turn % 2 == 0);
            }
        }
        // sequences that end at a tile's edge, and one at the matrix's last row
        std::vector<int> edges{0};
        for (int s = 0; s < 70; ++s) edges.push_back(edges.back() + bm * next(4) + (s % 9 == 0 ? 1 : 0));
        both(&edges, edges.back(), bm, 2, 2, true);
        // longer ones than are taken, and bounds outside the matrix
        std::vector<int> far{-50, 10, 900, 1 << 30};
        both(&far, 1000, bm, 2, 1, true, 333);
        for (int n : {4095, 4096, 4097, 10000})
            if (large || n < 4097 || bm == 64) {
                const auto off = offsets(n, 5, 4);
                both(&off, off.back() + 9, bm, 1, 1, true);
            }
        if (large) {
            const auto off = offsets(bm == 64 ? 300000 : 262145, 3, 5);
            both(&off, off.back() + 1, bm, 1, 1, true);
        }
    }
    std::printf("attention_index_check: %ld checks\n", checks);
    return 0;
}
